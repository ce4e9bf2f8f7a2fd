"""Log probabilities of given tokens, entropy, top alternatives and their
gradient, against the definitions in 64 bits (tests/loss_reference.py)."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo, losses
from tests import loss_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(n, v, dtype, seed=0, stride=None, offset=0, scale=3.0):
    """[n, v] logits, rows `stride` apart, starting `offset` elements into their buffer."""
    stride = stride or v
    buf = torch.full((offset + n * stride + 16,), 1e4, dtype=dtype, device="cuda")   # what lies between rows is not read as logits
    x = buf[offset:offset + n * stride].view(n, stride)[:, :v]
    x.copy_((torch.randn((n, v), generator=gen(seed), device="cuda") * scale).to(dtype))
    return x


def check_forward(x, tokens, k, temperature, **more):
    o = losses.token_logprobs(x, tokens, top_k=k, temperature=temperature, **more)
    n, v = x.shape
    d, p, lp, lnz = ref.row_stats(x, temperature)
    u = 2.0 ** -24
    tol = lambda dd: 2.0 ** -19 + 4 * u * (dd.abs().nan_to_num(0, 0, 0) + lnz.abs().nan_to_num(0, 0, 0))
    if tokens is not None:
        t = tokens[:, None]
        want = lp.gather(1, t.clamp(0, v - 1))
        want = torch.where(t < 0, torch.zeros_like(want), torch.where(t >= v, torch.full_like(want, math.nan), want))
        ref.close(o.logp[:, None], want, tol(d.gather(1, t.clamp(0, v - 1))), "logp")
    else:
        assert o.logp is None
    ed = torch.where(p == 0, torch.zeros_like(p), p * d).sum(1)
    h = torch.where((p.sum(1) == 0), torch.zeros_like(ed), ref.entropy(p, lp))
    ref.close(o.entropy, h, 2.0 ** -18 + 2.0 ** -19 * (lnz[:, 0].abs() + ed.abs()).nan_to_num(0, 0, 0), "entropy")
    if k:
        ids = ref.top(x, k)
        assert torch.equal(o.top_ids.long(), ids)
        ref.close(o.top_logp, lp.gather(1, ids), tol(d.gather(1, ids)), "top_logp")
    return o


SHAPES = [(1, 1, 1), (3, 2, 2), (1, 7, 3), (5, 31, 31), (2, 257, 128), (7, 1000, 5), (1, 4099, 20), (33, 8191, 64),
          (4, 50257, 20), (1, 50257, 128), (160, 50257, 1), (3, 128256, 64), (700, 12345, 17), (2, 262144, 100)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,v,k", SHAPES)
def test_forward(n, v, k, dtype):
    x = make(n, v, dtype, seed=n + v)
    t = torch.randint(0, v, (n,), generator=gen(1), device="cuda")
    check_forward(x, t, k, 1.0)
    check_forward(x, t, 0, 0.7)
    check_forward(x, None, k, 3.0)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("offset", [0, 1, 3, 5, 7, 8])
@pytest.mark.parametrize("stride", [0, 1, 7, 8])
def test_any_alignment_and_stride(stride, offset, dtype):
    v = 1003
    x = make(9, v, dtype, seed=offset, stride=v + stride, offset=offset)
    t = torch.randint(0, v, (9,), generator=gen(2), device="cuda")
    check_forward(x, t, 10, 1.0)
    check_grad(x, t, 10, 1.0)


@pytest.mark.parametrize("v", [50257 + i for i in range(17)] + [4096 * 8 + i for i in (-1, 0, 1)])
def test_every_row_end(v):
    x = make(5, v, BF, seed=v)
    x[:, -1] = 30.0                       # the last element matters
    x[1:, 0] = 31.0
    t = torch.full((5,), v - 1, device="cuda")
    check_forward(x, t, 3, 1.0)


def check_grad(x, tokens, k, temperature, seed=3, g=True, h=True, gt=True):
    n = x.shape[0]
    y = x.detach()
    leaf = y.requires_grad_(True) if y.is_leaf else y
    o = losses.token_logprobs(leaf, tokens, top_k=k, temperature=temperature)
    rnd = lambda *s: torch.randn(s, generator=gen(seed), device="cuda")
    outs, gs = [], []
    gl = ge = gtop = None
    if g and tokens is not None:
        gl = rnd(n)
        outs.append(o.logp), gs.append(gl)
    if h:
        ge = rnd(n) * 0.3
        outs.append(o.entropy), gs.append(ge)
    if gt and k:
        gtop = rnd(n, k) * 0.1
        outs.append(o.top_logp), gs.append(gtop)
    grad, = torch.autograd.grad(outs, leaf, gs)
    y.requires_grad_(False)
    want, scale = ref.logprobs_grad(x, temperature, tokens, gl, ge, o.top_ids, gtop)
    assert grad.shape == x.shape and grad.dtype == x.dtype
    ref.close(grad, want, ref.grad_tolerance(want, scale, x.dtype), "gradient")
    return grad


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,v,k", SHAPES)
def test_gradient(n, v, k, dtype):
    x = make(n, v, dtype, seed=n + v)
    t = torch.randint(0, v, (n,), generator=gen(1), device="cuda")
    check_grad(x, t, k, 1.0)
    check_grad(x, t, 0, 0.7, h=False)
    check_grad(x, None, k, 2.0)


def masked_rows(v, dtype):
    """Rows with everything that a mask may leave behind."""
    lowest = torch.finfo(dtype).min
    x = make(12, v, dtype, seed=11)
    x[0, :] = -INF                        # nothing left
    x[1, :] = -INF
    x[1, v // 2] = 1.0                    # one token left
    x[2, :] = lowest                      # masked by the lowest value: uniform
    x[3, :] = lowest
    x[3, 5] = 2.0
    x[4, :] = -INF
    x[4, [0, v - 1]] = lowest             # two tokens left, both at the lowest value
    x[5, 3] = math.nan
    x[6, 4] = INF
    x[7, v // 3:] = -INF                  # part of the vocabulary
    x[8, :] = 0.0
    x[8, ::2] = -0.0                      # one value, two signs
    x[9, :] = torch.finfo(dtype).max
    x[10, : v // 2] = lowest
    x[10, v // 2:] = torch.finfo(dtype).max / 2
    x[11, ::3] = lowest
    x[11, 1::3] = -INF
    return x


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("temperature", [1.0, 0.25, 8.0])
@pytest.mark.parametrize("v", [100, 1001, 50257])
def test_masks_and_special_values(v, temperature, dtype):
    x = masked_rows(v, dtype)
    t = torch.tensor([0, v // 2, 7, 5, v - 1, 2, 4, v - 1, 1, 3, v - 1, 0], device="cuda")
    keep = torch.tensor([i for i in range(12) if i not in (5, 6)], device="cuda")
    check_forward(x[keep], t[keep], 50, temperature)
    check_grad(x[keep], t[keep], 50, temperature)
    o = losses.token_logprobs(x, t, top_k=5, temperature=temperature)
    for r in (5, 6):                      # NaN and +inf: NaN all over the row, ids valid
        assert o.logp[r].isnan() and o.entropy[r].isnan() and o.top_logp[r].isnan().all()
        assert ((o.top_ids[r] >= 0) & (o.top_ids[r] < v)).all() and o.top_ids[r].unique().numel() == 5
    assert o.top_ids[5, 0] == 3 and o.top_ids[6, 0] == 4
    leaf = x.clone().requires_grad_(True)
    o = losses.token_logprobs(leaf, t, temperature=temperature)
    grad, = torch.autograd.grad(o.logp, leaf, torch.ones(12, device="cuda"))
    assert grad[5].isnan().all() and grad[6].isnan().all() and (grad[0] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [300, 20000, 128256])
@pytest.mark.parametrize("order", ["constant", "ascending", "descending", "few levels", "late", "one chunk"])
def test_top_of_awkward_orders(order, v, dtype):
    """Ties over the whole row, values that grow along it, and tops that lie together."""
    j = torch.arange(v, device="cuda", dtype=torch.float32)
    x = {"constant": j * 0 + 1.5, "ascending": j / v * 40, "descending": 20 - j / v * 40, "few levels": (j * 7919 % 5),
         "late": torch.where(j >= v - 150, 5.0 + j % 3, j * 0 - 2), "one chunk": torch.where((j > 130) & (j < 280), j % 11, -j % 2)}[order]
    x = torch.stack([x, x.flip(0), -x]).to(dtype)
    for k in (1, 20, 128):
        check_forward(x, torch.tensor([0, v - 1, v // 2], device="cuda"), k, 1.0)


def test_tokens_that_are_none_or_out_of_range():
    x = make(5, 1000, BF)
    t = torch.tensor([-1, 999, 1000, -100, 1 << 40], device="cuda")
    o = check_forward(x, t, 0, 1.0)
    assert o.logp[0] == 0 and o.logp[3] == 0
    grad = check_grad(x, t, 0, 1.0, h=False)
    assert (grad[0] == 0).all() and (grad[3] == 0).all() and grad[2].isnan().all() and grad[4].isnan().all()


def test_rows_without_an_incoming_gradient_are_not_read():
    x = make(4, 5001, F32)
    x[1] = math.nan
    x[2] = INF
    leaf = x.clone().requires_grad_(True)
    o = losses.token_logprobs(leaf, torch.zeros(4, dtype=torch.long, device="cuda"))
    w = torch.tensor([1.0, 0.0, 0.0, 2.0], device="cuda")
    grad, = torch.autograd.grad((o.logp, o.entropy), leaf, (w, w))
    assert (grad[1:3] == 0).all() and torch.isfinite(grad).all() and (grad[0] != 0).any()


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_batches_sliced_along_time(dtype):
    """logits[:, :-1] against tokens[:, 1:], read where they lie; and two transposed leading dimensions."""
    b, t, v = 3, 17, 1003
    full = (torch.randn((b, t, v), generator=gen(5), device="cuda") * 3).to(dtype)
    tokens = torch.randint(0, v, (b, t), generator=gen(6), device="cuda")
    g = torch.randn((b, t - 1), generator=gen(7), device="cuda")
    leaf = full.clone().requires_grad_(True)
    o = losses.token_logprobs(leaf[:, :-1], tokens[:, 1:], top_k=4, temperature=0.9)
    grad, = torch.autograd.grad(o.logp, leaf, g)
    flat = full[:, :-1].reshape(-1, v)
    d, p, lp, lnz = ref.row_stats(flat, 0.9)
    at = tokens[:, 1:].reshape(-1, 1)
    assert o.logp.shape == (b, t - 1) and o.top_ids.shape == (b, t - 1, 4)
    ref.close(o.logp.reshape(-1, 1), lp.gather(1, at), 2.0 ** -17, "logp")
    want, scale = ref.logprobs_grad(flat, 0.9, at[:, 0], g.reshape(-1))
    ref.close(grad[:, :-1].reshape(-1, v), want, ref.grad_tolerance(want, scale, dtype), "gradient")
    assert (grad[:, -1] == 0).all()
    swapped = losses.token_logprobs(full.transpose(0, 1)[:, :2], tokens.t()[:, :2], top_k=4, temperature=0.9)
    assert torch.equal(swapped.logp, losses.token_logprobs(full[:2].contiguous(), tokens[:2], temperature=0.9).logp.t())


def test_gradient_against_differences():
    """Central differences of the 32-bit forward pass itself."""
    n, v, k, eps = 3, 37, 5, 2.0 ** -6
    x = make(n, v, F32, seed=21, scale=1.5)
    t = torch.tensor([3, 36, 0], device="cuda")
    gl, ge, gt = (torch.randn(s, generator=gen(9), device="cuda") for s in ((n,), (n,), (n, k)))
    ids = losses.token_logprobs(x, t, top_k=k).top_ids

    def value(y):
        o = losses.token_logprobs(y, t)
        lp = losses.token_logprobs(y.repeat_interleave(k, 0), ids.reshape(-1).long()).logp.view(n, k)
        return (gl.double() * o.logp.double() + ge.double() * o.entropy.double()) + (gt.double() * lp.double()).sum(1)

    leaf = x.clone().requires_grad_(True)
    o = losses.token_logprobs(leaf, t, top_k=k)
    grad, = torch.autograd.grad((o.logp, o.entropy, o.top_logp), leaf, (gl, ge, gt))
    for j in range(v):
        e = torch.zeros_like(x)
        e[:, j] = eps
        num = (value(x + e) - value(x - e)) / (2 * eps)
        # third derivatives are of the size of the weights (below 8 together): eps^2/6 * 8 * a few;
        # roundings of values near 10: 2^-19 / eps
        assert (grad[:, j].double() - num).abs().max() < 4 * 8 * eps ** 2 / 6 + 16 * 2.0 ** -19 / eps


def test_in_place_gradient_and_overlap():
    x = make(6, 3001, BF, seed=4)
    t = torch.randint(0, 3001, (6,), generator=gen(1), device="cuda")
    g = torch.randn(6, generator=gen(2), device="cuda")
    stats = torch.empty(6, 4, device="cuda")
    fo.fo_token_logprobs(x, t, logp=torch.empty(6, device="cuda"), stats=stats)
    apart = torch.empty(6, 3001, dtype=BF, device="cuda")
    fo.fo_token_logprobs_grad(x, stats, apart, t, g)
    y = x.clone()
    fo.fo_token_logprobs_grad(y, stats, y, t, g)
    assert torch.equal(y, apart)
    buf = torch.empty(7, 3001, dtype=BF, device="cuda")
    with pytest.raises(fo.FoError, match="ALIAS"):
        fo.fo_token_logprobs_grad(buf[:6], stats, buf[1:], t, g)


def test_gradient_of_another_layout_than_the_logits():
    """Padded logits with a dense gradient and the reverse: rows of the two start at unlike alignments."""
    n, v = 11, 1003
    t = torch.randint(0, v, (n,), generator=gen(1), device="cuda")
    g = torch.randn(n, generator=gen(2), device="cuda")
    for dtype in (BF, F32):
        for ps, po in ((0, 0), (5, 0), (1, 3), (0, 1)):
            x = make(n, v, dtype, seed=8, stride=v + ps)
            stats = torch.empty(n, 4, device="cuda")
            fo.fo_token_logprobs(x, t, logp=torch.empty(n, device="cuda"), stats=stats)
            out = torch.full((n + 1, v + po), 7.0, dtype=dtype, device="cuda")
            fo.fo_token_logprobs_grad(x, stats, out[:n, :v], t, g)
            want, scale = ref.logprobs_grad(x, 1.0, t, g)
            ref.close(out[:n, :v], want, ref.grad_tolerance(want, scale, dtype), "gradient")
            assert (out[n] == 7).all() and (out[:, v:] == 7).all()      # nothing beyond the rows is written


def test_writes_stay_inside_their_arrays():
    n, v, k = 5, 777, 9
    x = make(n, v, BF)
    t = torch.zeros(n, dtype=torch.long, device="cuda")
    for cut in (1, 3):
        f = [torch.full((n * w + 8,), 7.0, device="cuda") for w in (1, 1, k)]
        ids = torch.full((n * k + 8,), 7, dtype=torch.int32, device="cuda")
        fo.fo_token_logprobs(x, t, k, f[0][cut:cut + n], f[1][cut:cut + n], ids[cut:cut + n * k], f[2][cut:cut + n * k])
        for a, w in zip(f + [ids], (1, 1, k, k)):
            assert (a[:cut] == 7).all() and (a[cut + n * w:] == 7).all() and (a[cut:cut + n * w] != 7).all() or w == k


def test_other_streams_graphs_and_repetition():
    """The call's own stream is used; a captured call replays on new logits; results repeat bit for bit."""
    x = make(64, 50257, BF, seed=1)
    t = torch.randint(0, 50257, (64,), generator=gen(1), device="cuda")
    want = losses.token_logprobs(x, t, top_k=8)
    for _ in range(3):
        again = losses.token_logprobs(x, t, top_k=8)
        assert all(torch.equal(a, b) for a, b in zip(want, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = x.clone()
        y.add_(1.0)
        y.sub_(1.0)
        got = losses.token_logprobs(x, t, top_k=8)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    z = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = losses.token_logprobs(z, t, top_k=8)
    z.copy_(x.flip(0))
    graph.replay()
    again = losses.token_logprobs(z, t, top_k=8)      # the rows at the same alignments: the same bits
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert torch.equal(out.top_ids, want.top_ids.flip(0))


def test_many_rows_and_offsets_beyond_32_bits():
    """More rows than a grid dimension of 65535, and elements past 2^32."""
    x = make(70001, 33, BF, seed=2)
    t = torch.randint(0, 33, (70001,), generator=gen(1), device="cuda")
    check_forward(x, t, 3, 1.0)
    check_grad(x, t, 0, 1.0)
    stride = (1 << 31) + 5                       # rows 4 GB apart: the third starts past 2^32 elements
    buf = torch.empty(2 * stride + 50257, dtype=BF, device="cuda")
    rows = torch.as_strided(buf, (3, 50257), (stride, 1))
    rows.copy_(make(3, 50257, BF, seed=3))
    check_forward(rows, torch.tensor([1, 50256, 7], device="cuda"), 5, 1.0)
    stats = torch.empty(3, 4, device="cuda")
    t3 = torch.tensor([1, 50256, 7], device="cuda")
    fo.fo_token_logprobs(rows, t3, logp=torch.empty(3, device="cuda"), stats=stats)
    want, scale = ref.logprobs_grad(rows, 1.0, t3, torch.ones(3, device="cuda"))
    fo.fo_token_logprobs_grad(rows, stats, rows, t3, torch.ones(3, device="cuda"))
    ref.close(rows, want, ref.grad_tolerance(want, scale, BF), "gradient")


def test_no_rows():
    o = losses.token_logprobs(torch.empty(0, 100, device="cuda"), torch.empty(0, dtype=torch.long, device="cuda"), top_k=3)
    assert o.logp.shape == (0,) and o.top_ids.shape == (0, 3)


def test_refusals():
    x = make(4, 100, BF)
    t = torch.zeros(4, dtype=torch.long, device="cuda")
    with pytest.raises(TypeError, match="logits"):
        losses.token_logprobs(x.double(), t)
    with pytest.raises(TypeError, match="tokens"):
        losses.token_logprobs(x, t.int())
    with pytest.raises(ValueError, match="tokens"):
        losses.token_logprobs(x, t[:3])
    with pytest.raises(ValueError, match="contiguous"):
        losses.token_logprobs(x.t(), torch.zeros(100, dtype=torch.long, device="cuda"))
    with pytest.raises(ValueError, match="top_k"):
        losses.token_logprobs(x, t, top_k=101)
    with pytest.raises(ValueError, match="top_k"):
        losses.token_logprobs(x, t, top_k=129)
    with pytest.raises(fo.FoError, match="BAD_ARG"):
        losses.token_logprobs(x, t, temperature=0.0)
    with pytest.raises(fo.FoError, match="SIZE"):
        losses.token_logprobs(torch.empty(1, fo.FO_MAX_ROW_BYTES // 4 + 1, device="cuda"), t[:1])
    with pytest.raises(ValueError, match="CUDA"):
        losses.token_logprobs(x.cpu(), t.cpu())
    with pytest.raises(ValueError, match="strides"):
        losses.token_logprobs(torch.empty(4, 6, 8, 10, device="cuda")[:3, :5, :7], torch.zeros(3, 5, 7, dtype=torch.long, device="cuda"))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("v,k", [(40, 40), (130, 64), (1000, 20), (1000, 65), (1000, 128), (4099, 64), (9001, 3), (33000, 64), (70001, 100)])
def test_many_rows_of_each_width(v, k, dtype):
    """Enough rows that each is one CTA's: of 64, 128 and 256 threads by its length and its list."""
    n = 640 if v > 20000 else 1500
    x = make(n, v, dtype, seed=v)
    x[7] = -INF                               # nothing left
    x[8, 2:] = -INF                           # fewer tokens left than are listed
    x[9] = 0.5                                # all tied
    x[10, ::2] = -0.0
    x[10, 1::2] = 0.0
    t = torch.randint(0, v, (n,), generator=gen(1), device="cuda")
    check_forward(x, t, k, 0.8)
    check_forward(x, t, 0, 1.0)


def test_alternatives_of_rows_with_nan():
    """NaN counts as the largest value, wherever it lies; the ids stay valid and distinct."""
    for n, v in ((2, 50257), (900, 1000)):
        x = make(n, v, BF, seed=v)
        x[0, [3, v // 2, v - 1]] = math.nan
        x[1, :] = math.nan
        o = losses.token_logprobs(x, top_k=10)
        assert o.top_ids[0, :3].tolist() == [3, v // 2, v - 1]
        assert o.top_ids[1].tolist() == list(range(10))
        assert o.top_ids[0].unique().numel() == 10 and o.top_logp[:2].isnan().all()


@pytest.mark.parametrize("k", [0, 1, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("n,v,dtype", [(100, 20001, BF), (300, 100003, F16), (761, 8192, BF), (1600, 16001, F32), (3100, 5003, BF), (1700, 70001, F16)])
def test_rows_shared_in_every_way(n, v, dtype, k):
    """Clusters and single CTAs of each width, lists below and above half of a CTA's threads."""
    x = make(n, v, dtype, seed=n + k)
    t = torch.randint(0, v, (n,), generator=gen(1), device="cuda")
    o = losses.token_logprobs(x, t, top_k=k, temperature=0.8)
    for i in range(0, n, 400):                # in parts, for the reference's 64-bit arrays
        at = slice(i, i + 400)
        d, p, lp, lnz = ref.row_stats(x[at], 0.8)
        tol = lambda dd: 2.0 ** -19 + 4 * 2.0 ** -24 * (dd.abs() + lnz.abs())
        one = t[at, None]
        ref.close(o.logp[at, None], lp.gather(1, one), tol(d.gather(1, one)), "logp")
        spread = (p * d).sum(1).abs()
        ref.close(o.entropy[at], ref.entropy(p, lp), 2.0 ** -18 + 2.0 ** -19 * (lnz[:, 0].abs() + spread), "entropy")
        if k:
            ids = ref.top(x[at], k)
            assert torch.equal(o.top_ids[at].long(), ids)
            ref.close(o.top_logp[at], lp.gather(1, ids), tol(d.gather(1, ids)), "top_logp")
