"""The teacher's distribution in the distillation losses: its precision, wherever its logits lie."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo, losses
from tests import loss_reference as ref
from tests.test_gpu_logprobs import gen

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


@pytest.mark.parametrize("temperature", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("shift", [0.0, 20.0, -100.0, 100.0, 1000.0, 30000.0])
@pytest.mark.parametrize("k", [2, 8, 64, 128])
def test_precision_does_not_depend_on_where_the_logits_lie(k, shift, temperature):
    """A student that is uniform over a power of two of tokens has exact probabilities, so that loss and gradient
    show the teacher's. Roundings (u = 2^-24), with d = (y - max) / T: an entry's d has 3 of |d|; its exponential 4
    (two ulp) more; the normaliser those of its terms, 3 E|d| + 4, and 9 chained additions, of which ln takes the same
    and 2 of its own size; q one reciprocal and one product. So q is within (3 |d| + 3 E|d| + 19) u, relatively, and
    ln q within (3 |d| + 3 E|d| + 13 + 2 ln z + |ln q|) u. The loss is a sum of products with ln V: 11 roundings of
    its terms' sizes."""
    v, n = 512, 64
    x = torch.zeros(n, v, device="cuda")
    ids = torch.rand((n, v), generator=gen(k), device="cuda").topk(k, dim=1).indices.to(torch.int32)
    # steps that FP32 holds beside the shift, so that the shifted logits are the same ones
    y = (torch.randn((n, k), generator=gen(k + 1), device="cuda") * 2 * 256).round() / 256 + shift
    want, grad, _, _ = ref.distill(x, ids, y, teacher_temperature=temperature)
    q, lq, _ = ref.teacher(ids, y, temperature)
    d = (y.double() - y.double().amax(1, keepdim=True)) / temperature
    spread = 3 * d.abs() + 3 * (q * d.abs()).sum(1, keepdim=True)
    off_q = (spread + 19) * U
    off_lq = (spread + 13 + 2 * math.log(k) + lq.abs()) * U
    terms = q * (lq.abs() + math.log(v))
    tol = (q * off_lq + terms * off_q + 11 * U * terms).sum(1)
    loss, g = losses.distill_loss_grad(x, ids, y, teacher_temperature=temperature)
    ref.close(loss, want, tol, "loss")
    allowed = torch.full_like(grad, 8 * U / v).scatter_add_(1, ids.long(), q * off_q)
    ref.close(g, grad, allowed + 2 * U * grad.abs(), "gradient")
    # the gradient of a row adds up to 0, as its roundings allow
    assert (g.double().sum(1).abs() <= (allowed + 2 * U * grad.abs()).sum(1)).all()


@pytest.mark.parametrize("temperature", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("shift", [0.0, 100.0, 1000.0])
def test_precision_with_a_tail(shift, temperature):
    """ln q = y / T - lse, the difference fused with the product by 1 / T in two parts: two roundings of its own size,
    and 2 u for the lower part. q has 4 u (two ulp) besides, the rest the sum of those and 9 additions."""
    v, n, k = 512, 64, 16
    x = torch.zeros(n, v, device="cuda")
    ids = torch.rand((n, v), generator=gen(k), device="cuda").topk(k, dim=1).indices.to(torch.int32)
    y = (torch.randn((n, k), generator=gen(k + 1), device="cuda") * 2 * 256).round() / 256 + shift
    lse = torch.logsumexp(y.double() / temperature, 1).float() + 0.3
    want, grad, _, _ = ref.distill(x, ids, y, teacher_temperature=temperature, tail=True, lse=lse)
    q, lq, rest = ref.teacher(ids, y, temperature, True, lse)
    off_lq = (2 * lq.abs() + 2) * U
    off_q = off_lq + 4 * U
    terms = q * (lq.abs() + math.log(v))
    off_rest = (q * off_q).sum(1) + 9 * U
    tol = (q * off_lq + terms * off_q + 11 * U * terms).sum(1) + off_rest * (2 + rest.log().abs() + math.log(v))
    loss, g = losses.distill_loss_grad(x, ids, y, teacher_temperature=temperature, tail=True, teacher_lse=lse)
    ref.close(loss, want, tol, "loss")
    allowed = (16 * U / v + off_rest / (v - k))[:, None].expand_as(grad).clone().scatter_add_(1, ids.long(), q * off_q)
    ref.close(g, grad, allowed + 2 * U * grad.abs(), "gradient")
