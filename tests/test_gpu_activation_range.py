"""Activations at the ends of their types' ranges: codes of the largest finite numbers, and functions of 16-bit types
where the exponential leaves FP32's normal numbers."""
import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo
from tests import act_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def finite_numbers(dtype):
    """Every finite 16-bit number; of FP32 the upper end, densely."""
    if dtype == F32:
        top = torch.arange(0x7f7fffff, 0x7f7fffff - 65536 * 31, -31, device="cuda", dtype=torch.int32).view(F32)
        return torch.cat([top, -top])
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    return x[torch.isfinite(x)]


@pytest.mark.parametrize("beside", [1, 7, 8, 40])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_finite_numbers_come_back_finite(dtype, beside):
    """Alone and beside smaller ones, in rows of vectors and in others: within half a step, as every other number."""
    x = finite_numbers(dtype)[:, None].repeat(1, beside)
    x[:, 1:] = x[:, 1:] * 0.5
    c = A.compress(x)
    y = A.expand(c)
    assert torch.isfinite(y).all()
    step = c.steps.double().repeat_interleave(32, 1)[:, :beside]
    unit = torch.maximum(x.double().abs() * 2 * ref.UNIT[dtype], torch.full_like(step, torch.finfo(dtype).smallest_normal * 2 * ref.UNIT[dtype]))
    # half a step, and a rounding to the type of a number at most a step larger
    assert ((y.double() - x.double()).abs() <= step * 0.5 * (1 + 2.0 ** -15) + (unit + step * 2 * ref.UNIT[dtype]) * 0.5).all()
    top = torch.finfo(dtype).max
    inside = ref.kept(x).abs() <= top
    assert torch.equal(y[inside], ref.kept(x).float().to(dtype)[inside])
    assert (y[~inside].abs() == top).all() and bool((~inside).any()) == (dtype != F32)   # FP32's stay within it


def test_numbers_beyond_a_smaller_type_are_infinite_in_it():
    """FP32 expanded to FP16: what no number of the group could have been is infinity, as in any conversion."""
    x = torch.tensor([[1e6, 60000.0, 65504.0, 80000.0, -1e6], [65504.0, -65504.0, 65300.0, 3.0, 0.0]], device="cuda")
    y = A.expand(A.compress(x), dtype=F16)
    assert torch.isinf(y[0, [0, 3, 4]]).all() and torch.isfinite(y[0, 1:3]).all()
    assert (y[1, :2].abs() == 65504.0).all() and torch.isfinite(y[1]).all()


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_gradients_beside_the_largest_numbers(dtype):
    top = torch.finfo(dtype).max
    x = torch.ones(4, 64, dtype=dtype, device="cuda")
    x[0, 0] = top
    w = torch.zeros(8, 64, dtype=dtype, device="cuda").requires_grad_(True)
    dy = torch.full((4, 8), 0.25, dtype=dtype, device="cuda")
    dy[0] = 0.0
    A.linear(x, w).backward(dy)
    assert torch.isfinite(w.grad).all() and ((w.grad[:, 0].double() / 0.75 - 1).abs() <= 2.0 ** -6).all()   # ones' codes: within 1 / 252
    # a gate and another half at the end of the range: products with a small gradient are numbers
    gate = torch.full((2, 40), top, dtype=dtype, device="cuda")
    y, kept = A.activation_forward(gate, "swiglu", up=gate.clone())
    dy = torch.full((2, 40), 2.0 ** -10, dtype=dtype, device="cuda")
    for g in A.activation_backward(kept, dy):
        assert torch.isfinite(g).all() and ((g.double() / (2.0 ** -10 * top) - 1).abs() <= 2.0 ** -6).all()


@pytest.mark.parametrize("w", [768, 20000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_beside_the_largest_numbers(dtype, w):
    x = torch.zeros(3, w, dtype=dtype, device="cuda")
    x[0, 5], x[1], x[2, 7] = torch.finfo(dtype).max, torch.finfo(dtype).max, 1.0
    dy = torch.full((3, w), 0.5, dtype=dtype, device="cuda")
    weight = torch.ones(w, device="cuda")
    _, kept = A.rms_norm_forward(x, weight)
    grad, gw = A.rms_norm_backward(kept, dy)
    want, tol, dw, dw_tol = ref.norm_backward(x, weight, 1e-6, dy)
    ref.close(grad, want, tol, "gradient")
    # r is a subnormal number of 21 bits here
    ref.close(gw, dw, dw_tol + 2.0 ** -21 * dw.abs(), "weight's gradient")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_far_negative_side_of_bfloat16(kind):
    """Results that are normal numbers keep their precision, to the last one (gelu's slope down to 2^-123: from 13.2 on,
    where its exponential is below 2^-126, it is 0)."""
    least, least_slope = (2.0 ** -133, 2.0 ** -133) if kind == "silu" else (2.0 ** -126, 2.0 ** -123)
    x = torch.arange(0x4000, 0x4340, device="cuda", dtype=torch.int32)      # 2 to 192, negative
    x = (x | 0x8000).to(torch.int16).view(BF)[:, None].contiguous()
    value, _, _, rel = ref.act(kind, x)
    y = A.activation(x, kind).double()
    # the function's own error, a rounding to BF16, and (silu) of numbers below 2^-126 a place of them
    assert ((y - value).abs() <= value.abs() * (rel + 2.0 ** -8 * (1 + 2.0 ** -8)) + least).all()
    _, kept = A.activation_forward(x, kind)
    got = A.activation_backward(kept, torch.ones_like(x)).double()
    _, slope, size, rel = ref.act(kind, ref.kept(x), BF)
    assert ((got - slope).abs() <= size * rel + slope.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + least_slope).all()
    normal = value.abs() >= 2.0 ** -126
    assert (y[normal] != 0).all() and normal.any()
