"""The losses over the whole range of finite logits and temperatures: masks that
are large finite numbers, rows far from zero, temperatures from 2^-20 to 2^20."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo, losses
from tests import loss_reference as ref
from tests.test_gpu_logprobs import check_forward, check_grad, gen

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def filled(v, dtype, fill, seed=0):
    """Rows with a large finite number where a mask or an offset would put it."""
    x = (torch.randn((8, v), generator=gen(seed), device="cuda") * 2).to(dtype)
    some = torch.randperm(v, generator=gen(seed + 1), device="cuda")[:max(1, v // 25)]
    x[0] = fill                                       # nothing else
    x[1] = fill
    x[1, v // 2] = 2.0                                # one token left
    x[2] = fill
    x[2, some] = x[7, some]                           # a few left, anywhere
    x[3, v // 2:] = fill                              # the upper half masked
    x[4, :3 * v // 4] = fill                          # what comes first masked
    x[5] = fill * (1 + torch.randint(0, 9, (v,), generator=gen(seed + 2), device="cuda") * float(torch.finfo(dtype).eps))
    x[6] = fill
    x[6, some] = fill * (1 - 0.125)                   # two large values
    return x


FILLS = [(BF, f) for f in (-1e4, -1e9, -1e10, -1e12, 1e10, 1e15)] + [(F32, f) for f in (-1e4, -1e9, -1e10, -1e12, 1e10, 1e15)] + \
        [(F16, -1e4), (F16, 6e4), (F16, -65504.0)]
TEMPERATURES = [1.0, 0.1, 1e-3, 2.0 ** -20, 300.0, 2.0 ** 20]


@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_logprobs_beside_large_finite_values(dtype, fill, temperature):
    for v, times in ((1003, 1), (1003, 100), (50257, 1)):
        x = filled(v, dtype, fill).repeat(times, 1)
        t = torch.randint(0, v, (x.shape[0],), generator=gen(4), device="cuda")
        t[1::8] = v // 2
        check_forward(x, t, 12, temperature)
        check_forward(x, t, 0, temperature)
        if times == 1 and (dtype != F16 or temperature >= 0.1):
            check_grad(x, t, 12, temperature)


def distill64(x, ids, y, temperature, tail, lse):
    """KL, its gradient by the logits, its tolerance and the scale of the gradient's terms, through
    logarithms: a rest of the student far below what 64 bits hold as a probability counts with its size."""
    d, p, lp, lnz = ref.row_stats(x, temperature)
    q, lq, rest = ref.teacher(ids, y, 1.0, tail, lse)
    at = ids.long()
    lp_at = lp.gather(1, at)
    loss = (q * (lq - lp_at)).sum(1)
    size = (q * (lq.abs() + lp_at.abs() + lnz.abs() + 1)).sum(1)
    target = torch.zeros_like(p).scatter_add_(1, at, q)
    grad, scale = p - target, p + target
    if tail:
        out = lp.scatter(1, at, -INF)
        lp_rest = torch.logsumexp(out, 1)
        loss = loss + rest * (rest.log() - lp_rest)
        size = size + rest * (rest.log().abs() + lp_rest.abs() + lnz[:, 0].abs() + 1) + 1
        share = (out - lp_rest[:, None]).exp()
        grad, scale = grad - share * rest[:, None], scale + share * (rest[:, None] + 1)
    return loss, grad / temperature, 2.0 ** -18 * (1 + size), scale / temperature


@pytest.mark.parametrize("temperature", TEMPERATURES)
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_distillation_beside_large_finite_values(dtype, fill, temperature):
    if dtype == F16 and temperature < 0.1:
        pytest.skip("gradients of 1 / T are beyond FP16")
    k = 7
    for v, times in ((1003, 1), (1003, 200), (50257, 1)):
        x = filled(v, dtype, fill).repeat(times, 1)
        n = x.shape[0]
        ids = torch.rand((n, v), generator=gen(5), device="cuda").topk(k, dim=1).indices.to(torch.int32)
        ids[::2, 0] = torch.where((ids[::2] == v // 2).any(1), ids[::2, 0], v // 2)
        y = torch.randn((n, k), generator=gen(6), device="cuda")
        lse = torch.logsumexp(y, 1) + 0.2
        for tail in (False, True):
            how = dict(temperature=temperature, tail=tail, teacher_lse=lse if tail else None)
            want, grad, tol, scale = distill64(x, ids, y, temperature, tail, lse if tail else None)
            loss, g = losses.distill_loss_grad(x, ids, y, **how)
            ref.close(loss, want, tol, "loss")
            ref.close(g, grad, ref.grad_tolerance(grad, scale, dtype), "gradient")
            leaf = x.detach().requires_grad_(True)
            alone = losses.distill_loss(leaf, ids, y, **how)
            ref.close(alone.detach(), want, tol, "loss alone")
            auto, = torch.autograd.grad(alone, leaf, torch.ones_like(alone))
            ref.close(auto, grad, ref.grad_tolerance(grad, scale, dtype), "gradient by automatic differentiation")


@pytest.mark.parametrize("temperature,first,then", [(83.0, -55840.0, -55584.0), (71.0, -57216.0, -56960.0), (78.0, -56416.0, -56160.0),
                                                    (63.0, -58112.0, -57856.0)])
def test_sums_carried_over_from_the_edge_of_fp16(temperature, first, then):
    """What a thread has summed beside a reference that is treated with care, FP16's lowest value being near, keeps its
    size when the reference moves to a number that needs none: (m - m') c, and not the difference of rounded products."""
    n, v = 310, 20000                         # one CTA of 256 threads a row
    x = torch.full((n, v), first, dtype=F16, device="cuda")
    x[:, 8192:8192 + 2048:8] = then           # one for each thread, after its first 32 elements
    check_forward(x, torch.full((n,), 8192, device="cuda"), 0, temperature)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("temperature", [1.0, 100.0, 4096.0, 2.0 ** 20])
def test_infinity_makes_the_row_nan_at_every_temperature(temperature, dtype):
    """Wherever +inf lies, first or last, and however far the reference may lie above the row's other logits."""
    v, most = 20001, 64500.0 if dtype == F16 else 1e6
    x = (torch.randn((6, v), generator=gen(3), device="cuda") * 2).to(dtype)
    x[3:] = most
    for r, at in enumerate((0, v // 2, v - 1) * 2):
        x[r, at] = INF
    t = torch.full((6,), 7, device="cuda")
    o = losses.token_logprobs(x, t, top_k=3, temperature=temperature)
    assert o.logp.isnan().all() and o.entropy.isnan().all() and o.top_logp.isnan().all()
    assert o.top_ids[:, 0].tolist() == [0, v // 2, v - 1] * 2
    ids = torch.tensor([[5, 6, 9]] * 6, dtype=torch.int32, device="cuda")
    y = torch.zeros(6, 3, device="cuda") - 2
    for tail in (False, True):
        loss, grad = losses.distill_loss_grad(x, ids, y, temperature=temperature, tail=tail)
        assert loss.isnan().all() and grad.isnan().all()
        assert losses.distill_loss(x, ids, y, temperature=temperature, tail=tail).isnan().all()
