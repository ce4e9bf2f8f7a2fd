"""The teacher's distribution in the distillation losses: its precision wherever its logits lie, and lists that
hold all that the teacher has."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo, losses
from tests import loss_reference as ref
from tests.test_gpu_logprobs import gen

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF, U = math.inf, 2.0 ** -24


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


@pytest.mark.parametrize("fill", [-INF, "lowest"])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_a_list_that_holds_all_that_a_mask_leaves(dtype, fill):
    """A grammar leaves fewer tokens than are listed, to the teacher and to the student: what the roundings of its log
    probabilities leave beside a sum of 1 is no mass, and the loss is not infinite for it."""
    fill = torch.finfo(dtype).min if fill == "lowest" else fill
    n, v, k = 400, 1003, 8
    live = torch.rand((n, v), generator=gen(1), device="cuda").topk(k, dim=1).indices
    left = 1 + torch.arange(n, device="cuda") % k                  # tokens that the mask leaves, 1 to k
    live = torch.where(torch.arange(k, device="cuda") < left[:, None], live, live[:, :1])
    rows = []
    for seed in (2, 3):
        x = torch.full((n, v), fill, dtype=dtype, device="cuda")
        rows.append(x.scatter_(1, live, (torch.randn((n, v), generator=gen(seed), device="cuda") * 2).to(dtype).gather(1, live)))
    told = losses.token_logprobs(rows[0], top_k=k)
    loss, grad = losses.distill_loss_grad(rows[1], told.top_ids, told.top_logp, tail=True)
    p = torch.softmax(rows[0].double(), 1)
    lp = torch.log_softmax(rows[1].double(), 1)
    want = torch.where(p > 0, p * (torch.log_softmax(rows[0].double(), 1) - lp), 0.0).sum(1)
    # each log probability within 2^-18 of its own, in the teacher's list and in the student's row
    assert ((loss.double() - want).abs() <= 2.0 ** -17 * (1 + (p * lp.abs().clamp(max=1e4)).sum(1))).all()
    assert torch.isfinite(grad.float()).all()
    alone = losses.distill_loss(rows[1], told.top_ids, told.top_logp, tail=True)
    assert ((alone - loss).abs() <= 2.0 ** -17 * (1 + loss.abs())).all()
    same, grad = losses.distill_loss_grad(rows[0], told.top_ids, told.top_logp, tail=True)
    assert same.abs().max() < 2.0 ** -16 and grad.float().abs().max() < 2.0 ** -16


def test_a_rest_that_the_student_excludes_is_infinite():
    """More than roundings leave: a teacher that holds tokens possible which the student excludes."""
    x = torch.full((3, 100), -INF, device="cuda")
    x[:, :2] = 0.0
    ids = torch.tensor([[0, 1]] * 3, dtype=torch.int32, device="cuda")
    y = torch.log(torch.tensor([[0.5, 0.4], [0.5, 0.4999], [0.5, 0.5]], device="cuda"))
    loss = losses.distill_loss(x, ids, y, tail=True)
    assert loss[:2].tolist() == [INF, INF] and abs(float(loss[2])) < 1e-6
