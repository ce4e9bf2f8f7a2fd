"""The policy loss on logits against 64 bits: loss, log probability and gradient, in one call and by automatic
differentiation."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo
from quantized_optimizer_state_gb300.losses import policy_loss, policy_loss_grad, token_logprobs
from tests import policy_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def make(n, v, dtype, seed=0, lo=0.2, hi=0.2, temperature=1.0):
    """Logits with likely tokens sampled, a policy that has moved (no ratio within 1e-3 of a border), advantages, a reference."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (3 * randn(n, v)).to(dtype)
    tokens = torch.randint(0, v, (n,), generator=g, device="cuda")
    x[torch.arange(n, device="cuda"), tokens] += (6 * torch.rand(n, generator=g, device="cuda")).to(dtype)
    l = torch.log_softmax(x.double() / temperature, 1).gather(1, tokens[:, None])[:, 0]
    moved = (0.3 * randn(n)).double()
    for border in (math.log(1 + hi), math.log(max(1 - lo, 1e-30))):
        moved = torch.where((moved - border).abs() < 1e-3, moved + 5e-3, moved)
    return x, tokens, (l - moved).float(), randn(n), (l + 0.3 * randn(n)).float(), (0.5 + torch.rand(n, generator=g, device="cuda"))


def check(x, tokens, old, adv, r=None, weight=None, what="", **how):
    n = x.shape[0]
    kw = dict(lo=how.get("clip_low", 0.2), hi=how.get("clip_high", 0.2), ref_logp=r, beta=how.get("kl_weight", 0.0),
              temperature=how.get("temperature", 1.0))
    o = policy_loss_grad(x, tokens, old, adv, ref_logp=r, row_weight=weight, **how)
    want = ref.policy(x, tokens, old, adv, weight=weight, **kw)
    for name, got, (value, tol) in zip(("loss", "log probability", "gradient"), o, want):
        ref.close(got, value, tol, f"{what}{name} in one call")
    # alone, and by automatic differentiation
    want = ref.policy(x, tokens, old, adv, **kw)
    alone = policy_loss(x, tokens, old, adv, ref_logp=r, **how)
    ref.close(alone.loss, *want[0], f"{what}loss")
    ref.close(alone.logp, *want[1], f"{what}log probability")
    leaf = x.detach().requires_grad_(True)
    p = policy_loss(leaf, tokens, old, adv, ref_logp=r, **how)
    assert not p.logp.requires_grad
    g = torch.ones(n, device="cuda") if weight is None else weight
    grad, = torch.autograd.grad(p.loss, leaf, g)
    value, tol = ref.policy(x, tokens, old, adv, weight=g, **kw)[2]
    ref.close(grad, value, tol, f"{what}gradient")
    return o


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,v", [(1, 1), (1, 7), (5, 33), (3, 777), (16, 50257), (2, 128256), (333, 1000), (1700, 260), (700, 30011),
                                 (40, 8191), (1, 200001)])
def test_against_64_bits(n, v, dtype):
    x, t, old, a, r, w = make(n, v, dtype, seed=v)
    check(x, t, old, a, weight=w / n)
    check(x, t, old, a, r, kl_weight=0.1)


@pytest.mark.parametrize("temperature", [0.3, 0.8, 2.5])
@pytest.mark.parametrize("lo,hi,beta", [(0.2, 0.28, 0.0), (0.0, 0.0, 0.05), (1.0, 5.0, 1.0), (0.5, 2.0 ** 90, 3.0)])
def test_settings(lo, hi, beta, temperature):
    x, t, old, a, r, w = make(200, 3001, BF, seed=7, lo=lo, hi=hi, temperature=temperature)
    check(x, t, old, a, r, w, clip_low=lo, clip_high=hi, kl_weight=beta, temperature=temperature)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_positions_that_are_none(dtype):
    x, t, old, a, r, w = make(300, 5003, dtype, seed=3)
    t[::3] = -1
    w[1::5] = 0.0
    t[7], w[7] = -2 ** 62, 1.0
    x[0], x[1] = NAN, INF                                        # rows that are not read
    w[1] = 0.0
    o = policy_loss_grad(x, t, old, a, ref_logp=r, kl_weight=0.1, row_weight=w)
    off = (t < 0) | (w == 0)
    assert (o.loss[off] == 0).all() and (o.logp[off] == 0).all() and (o.grad[off] == 0).all()
    assert (o.grad[~off] != 0).any(1).all() and torch.isfinite(o.grad).all()
    x[:2] = 0.0
    check(x, t, old, a, r, w, kl_weight=0.1)


@pytest.mark.parametrize("v,dtype", [(500, BF), (1500, BF), (3001, BF), (2000, F32), (9000, BF), (60000, BF)])
def test_padding_between_positions_changes_nothing(v, dtype):
    """Every path (rows in registers of a warp and of two, the ring, clusters): rows are the same bit for bit with
    padding before, between and after them as without."""
    n = 6000 if v < 5000 else 700
    x, t, old, a, r, w = make(n, v, dtype, seed=v)
    want = policy_loss_grad(x, t, old, a, ref_logp=r, kl_weight=0.1, row_weight=w)
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(3):
        off = torch.rand(n, generator=g, device="cuda") < 0.5
        tokens = torch.where(off, -1, t)
        for k in range(5):
            o = policy_loss_grad(x, tokens, old, a, ref_logp=r, kl_weight=0.1, row_weight=w)
            assert (o.loss[off] == 0).all() and (o.grad[off] == 0).all()
            assert all(torch.equal(p[~off], q[~off]) for p, q in zip(o, want))


@pytest.mark.parametrize("v", [700, 2500])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_special_values(dtype, v):
    n = 24
    x, t, old, a, r, w = make(n, v, dtype, seed=11)
    a = a.abs() + 0.1
    a[12:] *= -1
    x[0, 100:] = -INF
    t[0] = 5
    x[1], x[2, 3] = -INF, NAN                                    # no distribution; NaN
    x[3, 9] = INF
    x[4, t[4]] = -INF                                            # the sampled token is masked now
    x[5, t[5]] = torch.finfo(dtype).min
    t[6] = v                                                     # out of range
    t[7] = 2 ** 40
    old[8], old[9], old[10] = NAN, INF, -INF
    old[20], old[21] = -INF, INF                                 # advantage negative: no bound above
    a[11], old[11] = 0.0, -INF                                   # no policy term
    a[22], a[23] = NAN, INF
    x[13] = -INF
    x[13, t[13]] = 0.0                                           # one token left: l = 0
    x[14, t[14]] = -INF
    check(x, t, old, a, what="without KL: ")
    r = r.clone()
    r[15], r[16], r[17] = INF, -INF, NAN
    r[18] = 95.0                                                 # e^k beyond FP32
    check(x, t, old, a, r, kl_weight=0.1, what="with KL: ")


def test_the_border_counts_as_inside():
    x = torch.zeros(4, 2, device="cuda")
    x[:, 1] = -INF                                               # l = 0 exactly: the ratio is exp(-old)
    t = torch.zeros(4, dtype=torch.long, device="cuda")
    a = torch.tensor([1.0, -1.0, 1.0, -1.0], device="cuda")
    old = torch.zeros(4, device="cuda")
    x2 = torch.zeros(4, 2, device="cuda")                        # l = -ln 2
    o = policy_loss_grad(x, t, old, a, clip_low=0.0, clip_high=0.0)
    assert torch.equal(o.loss, -a) and (o.logp == 0).all() and (o.grad == 0).all()
    logp = token_logprobs(x2, t).logp
    o = policy_loss_grad(x2, t, logp, a, clip_low=0.0, clip_high=0.0)
    assert torch.equal(o.loss, -a) and torch.allclose(o.grad[:, 0], -0.5 * a, rtol=1e-6)
    out = policy_loss_grad(x2, t, logp - 0.01, a, clip_low=0.0, clip_high=0.0)   # above: only a negative advantage moves it
    assert (out.grad[::2] == 0).all() and (out.grad[1::2] != 0).all()


def test_small_kl_terms_keep_their_precision():
    """exp(k) - k - 1 for k where its terms cancel, with l exactly 0."""
    x = torch.full((200, 2), -INF, device="cuda")
    x[:, 0] = 0.0
    t = torch.zeros(200, dtype=torch.long, device="cuda")
    k = torch.cat([torch.logspace(-18, 1.9, 100, device="cuda"), -torch.logspace(-18, 6, 100, device="cuda")])
    o = policy_loss(x, t, torch.zeros(200, device="cuda"), torch.zeros(200, device="cuda"), ref_logp=k, kl_weight=1.0)
    kd = k.double()
    want = torch.where(kd.abs() < 1e-4, kd * kd / 2 * (1 + kd / 3 + kd * kd / 12), torch.expm1(kd) - kd)
    # a product, the series' or the exponential's 2 u and two differences, of terms at most 7 times the result beyond 1/2
    assert ((o.loss.double() - want).abs() <= 32 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all()


def test_large_masks_and_offsets():
    x, t, old, a, r, w = make(64, 1003, F32, seed=5)
    x[:, 500:] = -1e9
    t = t % 500
    old = token_logprobs(x, t, entropy=False).logp + 0.05
    check(x + 3e4, t, old, a, what="offset ")
    check(x, t, token_logprobs(x, t, temperature=2.0 ** -4, entropy=False).logp + 0.05, a, temperature=2.0 ** -4)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_layouts(dtype):
    n, v = 12, 1001
    x, t, old, a, r, w = make(n, v, dtype, seed=9)
    # sums follow the rows' alignment modulo 16 bytes, so that layouts agree within the tolerances
    loss, _, grad = ref.policy(x, t, old, a, weight=w)
    wide = torch.zeros(n, v + 7, dtype=dtype, device="cuda")
    wide[:, :v] = x
    o = policy_loss_grad(wide[:, :v], t, old, a, row_weight=w)
    ref.close(o.grad, *grad, "rows of a wider matrix")
    ref.close(o.loss, *loss, "loss")
    three = torch.zeros(3, 5, v, dtype=dtype, device="cuda")
    three[:, :4] = x.view(3, 4, v)
    cut = three[:, :-1]
    o = policy_loss_grad(cut, t.view(3, 4), old.view(3, 4), a.view(3, 4), row_weight=w.view(3, 4))
    assert o.loss.shape == (3, 4)
    ref.close(o.grad.reshape(n, v), *grad, "slice")
    same = policy_loss_grad(cut, t.view(3, 4), old.view(3, 4), a.view(3, 4), row_weight=w.view(3, 4), out=cut)
    assert same.grad is cut and torch.equal(cut.reshape(n, v), o.grad.reshape(n, v)) and (three[:, 4] == 0).all()
    leaf = three.clone().requires_grad_(True)
    leaf.data[:, :4] = x.view(3, 4, v)
    policy_loss(leaf[:, :-1], t.view(3, 4), old.view(3, 4), a.view(3, 4)).loss.backward(w.view(3, 4))
    assert (leaf.grad[:, 4] == 0).all()
    value, tol = ref.policy(x, t, old, a, weight=w)[2]
    ref.close(leaf.grad[:, :4].reshape(n, v), value, tol, "gradient of a slice")
    one = policy_loss(x[0], t[0], old[0], a[0])
    assert one.loss.shape == () and torch.equal(one.loss, policy_loss(x[:1], t[:1], old[:1], a[:1]).loss[0])
    none = policy_loss_grad(x[:0], t[:0], old[:0], a[:0])
    assert none.loss.shape == (0,) and none.grad.shape == (0, v)


@pytest.mark.parametrize("cut", [0, 1, 2, 3])
@pytest.mark.parametrize("n,v,dtype", [(5, 777, BF), (3, 128256, BF), (1, 50257, F32), (1300, 1000, BF), (500, 30011, F32), (4, 40, F32)])
def test_what_stands_around(n, v, dtype, cut):
    from tests.test_gpu_loss_guards import Guarded
    x, t, old, a, r, w = make(n, v, dtype, seed=v)
    loss, logp = Guarded(n, F32, cut), Guarded(n, F32, cut)
    grad, stats = Guarded(n * v, dtype, cut), Guarded(n * fo.FO_LOSS_STATS, F32, 0)
    fo.fo_policy_loss(x, t, old, a, r, w, loss.of, logp.of, stats.of, grad.of.view(n, v), kl_weight=0.1)
    for what, arr in (("loss", loss), ("logp", logp), ("gradient", grad), ("stats", stats)):
        arr.check(what)
    again = Guarded(n * v, dtype, cut)
    fo.fo_policy_loss_grad(x, t, stats.of, w, again.of.view(n, v))
    again.check("gradient from statistics")


def test_incoming_gradients_of_zero():
    x, t, old, a, r, w = make(9, 500, F32, seed=1)
    x[2] = NAN
    leaf = x.detach().requires_grad_(True)
    loss = policy_loss(leaf, t, old, a).loss
    g = torch.ones(9, device="cuda")
    g[2] = g[4] = 0.0
    grad, = torch.autograd.grad(loss, leaf, g)
    assert (grad[2] == 0).all() and (grad[4] == 0).all() and (grad[0] != 0).any()


def test_every_run_is_the_same():
    x, t, old, a, r, w = make(3000, 9000, BF, seed=2)
    first = policy_loss_grad(x, t, old, a, ref_logp=r, kl_weight=0.1, row_weight=w)
    for _ in range(5):
        o = policy_loss_grad(x, t, old, a, ref_logp=r, kl_weight=0.1, row_weight=w)
        assert all(torch.equal(p, q) for p, q in zip(o, first))


def test_gradient_against_differences():
    n, v = 6, 40
    x, t, old, a, r, w = make(n, v, F32, seed=4)
    how = dict(ref_logp=r, kl_weight=0.2, temperature=0.9)
    x = (x * 8).round() / 8
    grad = policy_loss_grad(x, t, old, a, **how).grad.double()
    f = lambda y: ref.policy(y, t, old, a, ref_logp=r, beta=0.2, temperature=0.9)[0][0].sum()
    h = 2.0 ** -10
    for i in range(n):
        for j in range(0, v, 7):
            up, down = x.double().clone(), x.double().clone()
            up[i, j] += h
            down[i, j] -= h
            # central differences: h^2 / 6 of a third derivative below 64, and the gradient's own 2^-18
            assert abs(float((f(up) - f(down)) / (2 * h) - grad[i, j])) <= 64 * h * h / 6 + 2.0 ** -16
