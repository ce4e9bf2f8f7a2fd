"""Distillation from a teacher's top logits: loss and gradient, against the
definitions in 64 bits (tests/loss_reference.py)."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo, losses
from tests import loss_reference as ref
from tests.test_gpu_logprobs import gen, make, masked_rows

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def make_teacher(n, v, k, seed=0, dtype=F32, short=True):
    """Distinct ids by row, some of them none (-1), and their logits; lse with a tail of a few percent."""
    g = gen(seed + 100)
    ids = torch.rand((n, v), generator=g, device="cuda").topk(min(k, v), dim=1).indices.to(torch.int32)
    if k > v:
        ids = torch.cat([ids, torch.full((n, k - v), -1, dtype=torch.int32, device="cuda")], 1)
    if short and n > 1:
        ids[n // 2, (k + 1) // 2:] = -1
    y = (torch.randn((n, k), generator=g, device="cuda") * 2).to(dtype)
    lse = torch.logsumexp(y.float(), 1) + 0.3 * torch.rand(n, generator=g, device="cuda") + 1e-3
    return ids, y, lse


def check(x, ids, y, lse=None, weight=None, temperature=1.0, teacher_temperature=1.0, tail=False):
    """The fused call, the loss alone, and the loss with its gradient by automatic differentiation."""
    how = dict(temperature=temperature, teacher_temperature=teacher_temperature, tail=tail, teacher_lse=lse)
    want, grad, tol, scale = ref.distill(x, ids, y, temperature, teacher_temperature, tail, lse, weight)
    loss, g = losses.distill_loss_grad(x, ids, y, row_weight=weight, **how)
    ref.close(loss, want, tol, "loss")
    ref.close(g, grad, ref.grad_tolerance(grad, scale, x.dtype), "gradient")
    leaf = x.detach()
    leaf.requires_grad_(True)
    alone = losses.distill_loss(leaf, ids, y, **how)
    w = torch.ones(x.shape[0], device="cuda") if weight is None else weight
    auto, = torch.autograd.grad(alone, leaf, w)
    leaf.requires_grad_(False)
    with torch.no_grad():
        assert torch.equal(losses.distill_loss(x, ids, y, **how).nan_to_num(-7), alone.nan_to_num(-7))
    use = w != 0
    full, _, tol1, _ = ref.distill(x, ids, y, temperature, teacher_temperature, tail, lse)
    ref.close(alone[use], full[use], tol1[use], "loss alone")
    ref.close(auto, grad, ref.grad_tolerance(grad, scale, x.dtype), "gradient by automatic differentiation")
    return loss, g


SHAPES = [(1, 1, 1), (3, 2, 2), (2, 5, 8), (5, 31, 4), (1, 300, 128), (7, 1000, 1), (1, 4099, 20), (33, 8191, 64),
          (4, 50257, 20), (1, 50257, 128), (170, 50257, 3), (3, 128256, 64), (700, 12345, 17), (2, 262144, 100)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,v,k", SHAPES)
def test_loss_and_gradient(n, v, k, dtype):
    x = make(n, v, dtype, seed=n + v)
    ids, y, lse = make_teacher(n, v, k, seed=v)
    w = torch.rand(n, generator=gen(5), device="cuda") + 0.1
    check(x, ids, y)
    check(x, ids, y, weight=w, temperature=2.0, teacher_temperature=2.0)
    check(x, ids, y, lse, w, temperature=0.7, tail=True)


@pytest.mark.parametrize("tdtype", [BF, F16, F32])
def test_teacher_types(tdtype):
    x = make(6, 1003, BF, seed=1)
    ids, y, _ = make_teacher(6, 1003, 33, dtype=tdtype)
    check(x, ids, y, teacher_temperature=3.0)
    lp = torch.log_softmax(y.float(), 1) - 0.1          # log probabilities with a rest of 10 %
    check(x, ids, lp.to(tdtype), tail=True)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("offset", [0, 1, 3, 5, 7, 8])
@pytest.mark.parametrize("stride", [0, 1, 7, 8])
def test_any_alignment_and_stride(stride, offset, dtype):
    v = 1003
    x = make(9, v, dtype, seed=offset, stride=v + stride, offset=offset)
    ids, y, lse = make_teacher(9, v, 12)
    check(x, ids, y)
    check(x, ids, y, lse, tail=True)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [100, 1001, 50257])
def test_masks_and_special_values(v, tail, dtype):
    x = masked_rows(v, dtype)
    ids, y, lse = make_teacher(12, v, 20, seed=3, short=False)
    check(x, ids, y, lse if tail else None, tail=tail)
    w = torch.ones(12, device="cuda")
    w[[0, 5, 6]] = 0.0                        # padding: whatever it holds
    loss, g = check(x, ids, y, lse if tail else None, w, tail=tail)
    assert (loss[[0, 5, 6]] == 0).all() and (g[[0, 5, 6]] == 0).all()


def test_teachers_with_odd_entries():
    v, n = 2000, 8
    x = make(n, v, F32, seed=6)
    ids, y, lse = make_teacher(n, v, 16, seed=2, short=False)
    ids[0] = -1                               # lists nothing
    y[1] = -INF                               # nothing of what it lists is possible
    y[2, 3:] = -INF
    ids[3, 1:] = ids[3, 0]                    # one id, listed 16 times
    ids[4, 8:] = ids[4, :8]                   # each twice
    y[5, 0] = 80.0                            # certain of one token
    x[6, ids[6].long()] = -INF                # the student excludes what the teacher lists
    check(x, ids, y)
    y[5, 0] = 5.0
    lse2 = torch.logsumexp(y.float(), 1).clamp(min=-1e4) + 0.05
    lse2[7] = lse2[7] - 0.2                   # more than the whole mass is listed: no rest
    check(x, ids, y, lse2, tail=True)
    x[7] = -INF
    x[7, ids[7].long()] = 1.0                 # the student leaves nothing for the rest
    lse2[7] = lse2[7] + 0.4
    check(x, ids, y, lse2, tail=True)


def test_ids_out_of_range_make_the_row_nan():
    x = make(4, 1000, BF)
    ids, y, lse = make_teacher(4, 1000, 8, short=False)
    ids[1, 3] = 1000
    ids[2, 0] = 2 ** 31 - 1
    for tail in (False, True):
        loss, g = check(x, ids, y, lse if tail else None, tail=tail)
        assert loss.isnan().tolist() == [False, True, True, False]
        assert g[1:3].isnan().all() and torch.isfinite(g[[0, 3]]).all()


@pytest.mark.parametrize("mass", [1e-2, 1e-5, 1e-7])
def test_rest_of_the_student_is_summed_not_subtracted(mass):
    """A student that leaves almost nothing outside the list: 1 - sum p would lose it."""
    v, k = 5000, 4
    x = torch.full((2, v), math.log(mass / (v - k)), device="cuda") + 0.1 * torch.randn((2, v), generator=gen(1), device="cuda")
    ids = torch.tensor([[0, 10, 100, 4999], [1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    x.scatter_(1, ids.long(), math.log(1 / k))
    y = torch.log(torch.tensor([[0.4, 0.3, 0.1, 0.1]] * 2, device="cuda"))
    loss, grad = losses.distill_loss_grad(x, ids, y, tail=True)
    want, g, tol, scale = ref.distill(x, ids, y, tail=True)
    ref.close(loss, want, tol, "loss")
    rest = g.clone()
    rest.scatter_(1, ids.long(), 0.0)         # unlisted: p (1 - r / p_rest), to 2^-17 of itself
    got = grad.double().scatter_(1, ids.long(), 0.0)
    assert ((got - rest).abs() <= 2.0 ** -17 * rest.abs()).all()


@pytest.mark.parametrize("gap", [60.0, 100.0, 300.0])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_rest_far_below_the_listed_logits(gap, dtype):
    """A rest whose probability FP32 cannot hold still has a finite loss and its own share of the gradient."""
    v = 3001
    x = make(2, v, dtype, seed=3, scale=1.0)
    x.sub_(gap / 2)
    ids = torch.tensor([[0, 10, 100, 3000], [1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    x.scatter_(1, ids.long(), gap / 2)
    y = torch.log(torch.tensor([[0.4, 0.3, 0.1, 0.1]] * 2, device="cuda"))
    loss, grad = check(x, ids, y, tail=True)
    assert torch.isfinite(loss).all() and (loss > 0.05 * gap).all()
    rest = grad.double().scatter_(1, ids.long(), 0.0).sum(1)     # minus what the teacher leaves for the rest
    assert (rest + 0.1).abs().max() < 0.1 * (2.0 ** -8 if dtype != F32 else 2.0 ** -17)


def test_gradient_against_differences():
    n, v, k, eps = 3, 41, 6, 2.0 ** -6
    x = make(n, v, F32, seed=21, scale=1.5)
    ids, y, lse = make_teacher(n, v, k, seed=4)
    for how in (dict(temperature=2.0, teacher_temperature=2.0), dict(tail=True, teacher_lse=lse)):
        _, grad = losses.distill_loss_grad(x, ids, y, **how)
        for j in range(v):
            e = torch.zeros_like(x)
            e[:, j] = eps
            num = (losses.distill_loss(x + e, ids, y, **how).double() - losses.distill_loss(x - e, ids, y, **how).double()) / (2 * eps)
            # third derivatives are at most 1; roundings of values below 8: 2^-19 / eps
            assert (grad[:, j].double() - num).abs().max() < eps ** 2 + 8 * 2.0 ** -19 / eps


def test_gradient_in_place_and_out():
    x = make(9, 50257, BF, seed=4)
    ids, y, lse = make_teacher(9, 50257, 50)
    loss, want = losses.distill_loss_grad(x, ids, y, tail=True, teacher_lse=lse)
    z = x.clone()
    loss2, got = losses.distill_loss_grad(z, ids, y, tail=True, teacher_lse=lse, out=z)
    assert got.data_ptr() == z.data_ptr() and torch.equal(z, want) and torch.equal(loss, loss2)
    stats = torch.empty(9, 4, device="cuda")
    fo.fo_distill(x, ids, y, lse, stats=stats, tail=True)
    z = x.clone()
    fo.fo_distill_grad(z, ids, y, stats, torch.ones(9, device="cuda"), z, lse, tail=True)
    assert torch.equal(z, want)
    out = torch.full((9, 50260), 7.0, dtype=BF, device="cuda")       # rows at another alignment than the logits'
    losses.distill_loss_grad(x, ids, y, tail=True, teacher_lse=lse, out=out[:, 1:50258])
    assert torch.equal(out[:, 1:50258], want) and (out[:, 0] == 7).all() and (out[:, 50258:] == 7).all()
    buf = torch.empty(10, 50257, dtype=BF, device="cuda")
    with pytest.raises(fo.FoError, match="ALIAS"):
        losses.distill_loss_grad(buf[:9], ids, y, out=buf[1:])


def test_batches_sliced_along_time():
    b, t, v, k = 3, 17, 1003, 9
    full = (torch.randn((b, t, v), generator=gen(5), device="cuda") * 3).to(BF)
    ids, y, _ = make_teacher(b * (t - 1), v, k)
    loss, g = losses.distill_loss_grad(full[:, :-1], ids.view(b, t - 1, k), y.view(b, t - 1, k))
    want, grad, tol, scale = ref.distill(full[:, :-1].reshape(-1, v), ids, y)
    assert loss.shape == (b, t - 1) and g.shape == (b, t - 1, v)
    ref.close(loss.view(-1), want, tol, "loss")
    ref.close(g.view(-1, v), grad, ref.grad_tolerance(grad, scale, BF), "gradient")
    last = full[:, -1].clone()
    losses.distill_loss_grad(full[:, :-1], ids.view(b, t - 1, k), y.view(b, t - 1, k), out=full[:, :-1])
    assert torch.equal(full[:, :-1], g) and torch.equal(full[:, -1], last)


def test_many_rows():
    x = make(70001, 33, BF, seed=2)
    ids, y, lse = make_teacher(70001, 33, 5)
    check(x, ids, y, lse, tail=True)


def test_streams_graphs_and_repetition():
    x = make(40, 50257, BF, seed=1)
    ids, y, lse = make_teacher(40, 50257, 30)
    how = dict(tail=True, teacher_lse=lse)
    want = losses.distill_loss_grad(x, ids, y, **how)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, losses.distill_loss_grad(x, ids, y, **how)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = losses.distill_loss_grad(x, ids, y, **how)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    z = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad = losses.distill_loss_grad(z, ids, y, **how)
    z.add_(0.5)
    graph.replay()
    again = losses.distill_loss_grad(z, ids, y, **how)
    assert torch.equal(loss, again[0]) and torch.equal(grad, again[1])


def test_alternatives_of_a_teacher_feed_a_student():
    """What token_logprobs writes down is what distill_loss reads: a student equal to the teacher has loss 0."""
    x = make(20, 5003, BF, seed=9)
    o = losses.token_logprobs(x, top_k=64, temperature=1.5)
    loss, grad = losses.distill_loss_grad(x, o.top_ids, o.top_logp, temperature=1.5, tail=True)
    assert loss.abs().max() < 2.0 ** -17
    assert grad.float().abs().max() < 2.0 ** -17
    plain = losses.distill_loss(x, o.top_ids, o.top_logp, temperature=1.5)
    assert (plain > 0).all()                  # the student spreads mass over what is not listed


def test_no_rows():
    e = torch.empty(0, 100, device="cuda")
    loss, grad = losses.distill_loss_grad(e, torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, 3, device="cuda"))
    assert loss.shape == (0,) and grad.shape == (0, 100)


def test_refusals():
    x = make(4, 1000, BF)
    ids, y, lse = make_teacher(4, 1000, 8)
    with pytest.raises(TypeError, match="teacher_ids"):
        losses.distill_loss(x, ids.long(), y)
    with pytest.raises(TypeError, match="teacher_logits"):
        losses.distill_loss(x, ids, y.double())
    with pytest.raises(ValueError, match="leading shape"):
        losses.distill_loss(x, ids[:3], y[:3])
    with pytest.raises(ValueError, match="128"):
        losses.distill_loss(x, ids.repeat(1, 17), y.repeat(1, 17))
    with pytest.raises(ValueError, match="tail"):
        losses.distill_loss(x, ids, y, teacher_lse=lse)
    with pytest.raises(ValueError, match="teacher_lse"):
        losses.distill_loss(x, ids, y, tail=True, teacher_lse=lse[:3])
    with pytest.raises(ValueError, match="row_weight"):
        losses.distill_loss_grad(x, ids, y, row_weight=lse[:3])
    with pytest.raises(TypeError, match="grad"):
        losses.distill_loss_grad(x, ids, y, out=torch.empty(4, 1000, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        losses.distill_loss_grad(x, ids, y, out=torch.empty(4, 999, dtype=BF, device="cuda"))
    with pytest.raises(fo.FoError, match="BAD_ARG"):
        losses.distill_loss(x, ids, y, temperature=-1.0)
    with pytest.raises(fo.FoError, match="BAD_ARG"):
        losses.distill_loss(x, ids, y, teacher_temperature=float("nan"))
    with pytest.raises(fo.FoError, match="BAD_ARG"):       # rows of the gradient on top of one another
        losses.distill_loss_grad(x, ids, y, out=torch.empty(1000, dtype=BF, device="cuda").expand(4, 1000))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v,dtype", [(2003, BF), (4100, F32), (33001, F16)])
def test_rows_that_a_cluster_takes_in_turn(v, dtype, tail):
    """More rows than CTAs: several by each, rows of weight 0 among them, in place and not."""
    n = 4000 if v < 10000 else 2500
    x = make(n, v, dtype, seed=v)
    ids, y, lse = make_teacher(n, v, 24, seed=5)
    ids[::7, 20] = ids[::7, 3]                # a token listed twice
    w = torch.rand(n, generator=gen(5), device="cuda") / n
    w[torch.rand(n, generator=gen(6), device="cuda") < 0.4] = 0.0
    x[w == 0] = math.nan
    how = dict(tail=tail, teacher_lse=lse if tail else None)
    want, grad, tol, scale = ref.distill(x.nan_to_num(0.0), ids, y, tail=tail, lse=how["teacher_lse"], weight=w)
    loss, g = losses.distill_loss_grad(x, ids, y, row_weight=w, **how)
    ref.close(loss, want, tol, "loss")
    ref.close(g, grad, ref.grad_tolerance(grad, scale, dtype), "gradient")
    for _ in range(2):
        z = x.clone()
        again, gz = losses.distill_loss_grad(z, ids, y, row_weight=w, out=z, **how)
        assert torch.equal(gz, g) and torch.equal(again, loss)
    keep = w != 0
    alone = losses.distill_loss(x[keep], ids[keep], y[keep], tail=tail, teacher_lse=lse[keep] if tail else None)
    ref.close(alone * w[keep], want[keep], tol[keep] * 1.01 + 2.0 ** -23 * want[keep].abs(), "loss alone")


def test_a_teacher_that_is_not_a_number():
    x = make(4, 1000, F32)
    ids, y, lse = make_teacher(4, 1000, 8, short=False)
    y[1, 2] = math.nan
    y[2, 5] = math.nan
    ids[2, 5] = -1                            # no entry: what stands beside it does not matter
    y[3, 0] = INF
    for tail in (False, True):
        loss, g = losses.distill_loss_grad(x, ids, y, tail=tail, teacher_lse=lse if tail else None)
        assert loss.isnan().tolist() == [False, True, False, True]
        assert g[1].isnan().all() and g[3].isnan().all() and torch.isfinite(g[[0, 2]]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_lists_with_tokens_listed_twice(dtype):
    """128 ids, some of them twice or three times, close together and far apart in the list; a row a CTA."""
    n, v = 600, 5003
    x = make(n, v, dtype, seed=8)
    ids, y, _ = make_teacher(n, v, 128, seed=8, short=False)
    for r, (to, of) in enumerate([(slice(96, 128), slice(0, 32)), (40, 3), (slice(1, 128, 2), slice(0, 128, 2)),
                                  ([10, 42, 74, 106], [10] * 4), ([32, 64], [0, 0]), (33, 32)]):
        ids[r::7, to] = ids[r::7, of].clone()
    x.scatter_(1, ids.clamp(min=0).long(), torch.full_like(y, 16.0).to(dtype))     # a listed token weighs as much as all others
    lse = torch.logsumexp(y, 1) + 0.2
    check(x, ids, y)
    check(x, ids, y, lse, tail=True)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("n,v,dtype", [(40, 16385, F32), (180, 200003, BF), (310, 128256, F16), (330, 80000, BF), (470, 50257, BF),
                                       (500, 130001, F32), (1300, 20011, F16), (4000, 60011, BF)])
def test_rows_shared_and_taken_in_every_way(n, v, dtype, tail):
    """One CTA a row, clusters, all rows in one turn or a few, two CTAs to an SM and three."""
    x = make(n, v, dtype, seed=n)
    ids, y, lse = make_teacher(n, v, 40, seed=v)
    w = torch.rand(n, generator=gen(5), device="cuda") / n
    w[::5] = 0.0
    how = dict(tail=tail, teacher_lse=lse if tail else None, temperature=1.3)
    loss, g = losses.distill_loss_grad(x, ids, y, row_weight=w, **how)
    alone = losses.distill_loss(x, ids, y, **how)
    for i in range(0, n, 250):                # in parts, for the reference's 64-bit arrays
        at = slice(i, i + 250)
        part = (x[at], ids[at], y[at], 1.3, 1.0, tail, lse[at] if tail else None)
        want, grad, tol, scale = ref.distill(*part, w[at])
        ref.close(loss[at], want, tol, "loss")
        ref.close(g[at], grad, ref.grad_tolerance(grad, scale, dtype), "gradient")
        want, _, tol, _ = ref.distill(*part)
        ref.close(alone[at], want, tol, "loss alone")
