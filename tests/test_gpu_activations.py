"""Activations kept in 8 bits: codes against their definition bit for bit, activation functions and norms against
64 bits, forward and backward."""
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo
from tests import act_reference as ref

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def make(shape, dtype, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    channel = torch.exp(torch.randn(shape[-1], generator=g, device="cuda"))
    return (x * channel * scale).to(dtype)


def placed(x, cut, pad):
    """The same values `cut` elements off a 16-byte boundary, rows `pad` elements apart."""
    n, w = x.shape
    buf = torch.full((cut + n * (w + pad) + 8,), 3.0, dtype=x.dtype, device="cuda")
    y = buf[cut:cut + n * (w + pad)].view(n, w + pad)[:, :w]
    return y.copy_(x)


def same(a, b):
    """Equal bit for bit, NaN for NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())


def check_codes(x, c, what="codes"):
    code, step = ref.codes(x)
    there = ~torch.isnan(step)
    assert torch.equal(torch.isnan(c.steps), ~there), f"{what}: steps that are NaN"
    assert torch.equal(c.steps.double()[there], step[there]), f"{what}: steps"
    wide = there.repeat_interleave(32, -1)
    assert torch.equal(c.codes.double()[wide], code[wide]), f"{what}: codes"


SIZES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 64), (7, 100), (1, 4096), (33, 768), (64, 257), (300, 1000), (1000, 40), (17, 16385)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,w", SIZES)
def test_codes(n, w, dtype):
    x = make((n, w), dtype, seed=w)
    c = A.compress(x)
    check_codes(x, c)
    assert c.codes.shape == (n, -(-w // 32) * 32) and c.steps.dtype == BF and c.dtype == dtype
    for to in (BF, F16, F32):
        assert torch.equal(A.expand(c, dtype=to), ref.kept(x).to(F32).to(to))   # exact in FP32, then one rounding
    assert A.expand(c).dtype == dtype


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("cut,pad", [(0, 8), (1, 0), (3, 5), (4, 4), (0, 1), (8, 24)])
@pytest.mark.parametrize("n,w", [(5, 96), (37, 1000), (4, 77)])
def test_codes_of_rows_anywhere(n, w, cut, pad, dtype):
    x = make((n, w), dtype, seed=cut)
    y = placed(x, cut, pad)
    c = A.compress(y)
    check_codes(x, c)
    back = placed(torch.zeros_like(x), cut, pad)
    around = back._base.clone()
    assert A.expand(c, out=back) is back
    assert torch.equal(back, ref.kept(x).to(F32).to(dtype))
    back.zero_()
    assert torch.equal(back._base, around)                       # nothing beside the rows


def test_ties_steps_and_extremes():
    x = torch.zeros(12, 64, device="cuda")
    x[0, :33] = torch.arange(33, device="cuda") + 0.5            # halves, step 1 is not reached: a = 32.5
    x[1, 0], x[1, 1:6] = 127.0, torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5], device="cuda")   # step 1: ties to even
    x[2, 0] = torch.finfo(F32).max
    x[3, 0], x[3, 1] = 2.0 ** -149, -2.0 ** -130
    x[4, 0], x[4, 1] = 127 * 2.0 ** -126, 2.0 ** -127
    x[5, 0] = 127.0 + 2.0 ** -17                                 # just above: the next step
    x[6, 0] = 127.0 - 2.0 ** -17
    x[7, 0], x[7, 40] = NAN, 1.0
    x[8, 1], x[8, 40] = INF, 1.0
    x[9, 2], x[9, 40] = -INF, -1.0
    x[10] = -0.0
    x[11, 5] = 1.0 / 3
    c = A.compress(x)
    check_codes(x, c)
    assert c.codes[1, :6].tolist() == [127, 0, 2, 2, 0, -2] and c.steps[1, 0] == 1.0
    y = A.expand(c)
    assert torch.isnan(y[7:10, :32]).all() and torch.isfinite(y[7:10, 32:]).all()
    assert (y[10] == 0).all() and y[8, 40] != 0
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(ref.kept(x).float()))
    for dtype in (BF, F16):                                      # every number of a type, as the largest and beside one
        every = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
        for x in (every[:, None].contiguous(), torch.cat([every.view(-1, 32), every.flip(0).view(-1, 32)], 1)):
            check_codes(x, A.compress(x), str(dtype))


def test_every_step_of_fp32_border():
    """Largest magnitudes next to 127 times a BF16 number: the smallest step that is enough, whatever the rounding."""
    s = (torch.arange(0x0080, 0x7c00, 7, device="cuda", dtype=torch.int32) << 16).view(F32).double() * 127
    a = s.float()
    a = a[torch.isfinite(a)]
    x = torch.stack([a, torch.nextafter(a, a * 0), torch.nextafter(a, a * 2)], 1).reshape(-1, 1).contiguous()
    check_codes(x, A.compress(x))


def test_codes_beyond_the_width_are_zero_and_leading_dimensions():
    x = make((2, 3, 45), BF)
    c = A.compress(x)
    assert c.codes.shape == (2, 3, 64) and c.steps.shape == (2, 3, 2)
    assert (c.codes[..., 45:] == 0).all()
    assert torch.equal(A.expand(c), ref.kept(x).to(BF))
    v = x[:, 1]                                                  # rows 3 * 45 apart
    assert torch.equal(A.expand(A.compress(v)), ref.kept(v).to(BF))
    e = x[:1, :1].expand(1, 5, 45)                               # one row read five times
    assert torch.equal(A.expand(A.compress(e)), ref.kept(e).to(BF))
    one = A.compress(x[0, 0])
    assert one.codes.shape == (64,) and torch.equal(A.expand(one), ref.kept(x[0, 0]).to(BF))
    none = A.compress(x[:0])
    assert none.codes.shape == (0, 3, 64) and A.expand(none).shape == (0, 3, 45)


def test_offsets_beyond_32_bits():
    n, w = 70000, 32768                                          # 2.3e9 elements
    x = torch.zeros((n, w), dtype=BF, device="cuda")
    rows = torch.tensor([0, 1, 32767, 65535, 65536, 69999], device="cuda")
    x[rows] = make((len(rows), w), BF)
    c = A.compress(x)
    assert torch.equal(c.codes[rows].double(), ref.codes(x[rows])[0])
    del x
    y = A.expand(c)
    assert torch.equal(y[rows], A.expand(A.Compressed(c.codes[rows], c.steps[rows], w, BF)))
    assert int((y != 0).any(1).sum()) == len(rows)


# --- activation functions -----------------------------------------------------------------------

def halves(x):
    w = x.shape[-1] // 2
    return x[..., :w], x[..., w:]


def check_activation(x, kind, dy, what=""):
    y, kept = A.activation_forward(x, kind)
    grad = A.activation_backward(kept, dy)
    gated = kind in ("swiglu", "geglu")
    a, b = halves(x) if gated else (x, None)
    want, tol = ref.forward(kind, a, b)
    ref.close(y, want, tol, f"{what}{kind} value")
    if not gated:
        want, tol = ref.backward(kind, a, dy)
        ref.close(grad, want, tol, f"{what}{kind} gradient")
    else:
        g, gt, h, ht = ref.backward(kind, a, dy, b)
        ref.close(halves(grad)[0], g, gt, f"{what}{kind} gate's gradient")
        ref.close(halves(grad)[1], h, ht, f"{what}{kind} other half's gradient")
    assert same(A.activation(x, kind), y)                 # the same without anything kept
    return y, kept, grad


@pytest.mark.parametrize("kind", list(A.KINDS))
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,w", [(1, 1), (3, 33), (2, 64), (16, 1000), (64, 257), (1000, 40), (5, 14336), (301, 2731)])
def test_activation(n, w, dtype, kind):
    gated = kind in ("swiglu", "geglu")
    x = make((n, 2 * w if gated else w), dtype, seed=w)
    check_activation(x, kind, make((n, w), dtype, seed=w + 1, scale=0.1))


@pytest.mark.parametrize("kind", list(A.KINDS))
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("cut,pad,w", [(0, 8, 96), (1, 0, 96), (3, 5, 100), (4, 12, 52), (0, 0, 36), (8, 8, 4096)])
def test_activation_of_rows_anywhere(cut, pad, w, dtype, kind):
    gated, n = kind in ("swiglu", "geglu"), 11
    x = make((n, 2 * w if gated else w), dtype, seed=w)
    dy = make((n, w), dtype, seed=w + 1, scale=0.1)
    y, kept, grad = check_activation(x, kind, dy)
    y2, kept2, grad2 = check_activation(placed(x, cut, pad), kind, placed(dy, cut, pad))
    assert torch.equal(y, y2) and torch.equal(grad, grad2)
    for p, q, half in zip(kept.inputs(), kept2.inputs(), halves(x) if gated else (x,)):
        check_codes(half, p)
        assert torch.equal(p.codes, q.codes) and torch.equal(p.steps, q.steps)
    if gated:
        a, b = halves(placed(x, cut, pad))
        y3, kept3 = A.activation_forward(a, kind, up=b.contiguous())
        g3, u3 = A.activation_backward(kept3, dy)
        assert torch.equal(y3, y) and torch.equal(torch.cat([g3, u3], 1), grad)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_activation_of_every_number(kind, dtype):
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype).view(-1, 32)
    want, tol = ref.forward(kind, x)
    ref.close(A.activation(x, kind), want, tol, kind)
    alone = x.reshape(-1, 1).contiguous()                        # a group each: the slope at every number's code
    _, kept = A.activation_forward(alone, kind)
    dy = torch.ones_like(alone)
    want, tol = ref.backward(kind, alone, dy)
    ref.close(A.activation_backward(kept, dy), want, tol, kind + " slope")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_of_fp32_far_out(kind):
    x = torch.cat([torch.linspace(-130, 130, 200001, device="cuda"), -torch.logspace(-44, 38, 50000, device="cuda"),
                   torch.logspace(-44, 38, 50000, device="cuda")])
    x = x[:x.numel() // 32 * 32].view(-1, 32).contiguous()
    want, tol = ref.forward(kind, x)
    ref.close(A.activation(x, kind), want, tol, kind)
    alone = x.reshape(-1, 1).contiguous()
    _, kept = A.activation_forward(alone, kind)
    want, tol = ref.backward(kind, alone, torch.ones_like(alone))
    ref.close(A.activation_backward(kept, torch.ones_like(alone)), want, tol, kind + " slope")


@pytest.mark.parametrize("kind", list(A.KINDS))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_activation_of_infinities_and_nan(kind, dtype):
    gated = kind in ("swiglu", "geglu")
    w = 128
    x = make((6, 2 * w if gated else w), dtype)
    x[0, 3], x[1, 40], x[2, 70], x[3, 100] = NAN, INF, -INF, 0.0
    if gated:
        x[4, w + 5], x[5, w + 37] = INF, NAN
    check_activation(x, kind, make((6, w), dtype, seed=1))


def test_incoming_gradients_in_other_layouts():
    x = make((6, 64), BF)
    y, kept = A.activation_forward(x, "silu")
    ones = torch.ones(1, 1, dtype=BF, device="cuda").expand(6, 64)
    want = A.activation_backward(kept, torch.ones_like(y))
    assert torch.equal(A.activation_backward(kept, ones), want)
    assert torch.equal(A.activation_backward(kept, torch.ones(64, 6, dtype=BF, device="cuda").t()), want)


# --- norm -----------------------------------------------------------------------------------------

def check_norm(x, weight, dy, eps=1e-6):
    y, kept = A.rms_norm_forward(x, weight, eps=eps)
    grad, grad_weight = A.rms_norm_backward(kept, dy)
    want, tol, r = ref.norm(x, weight, eps)
    ref.close(y, want, tol, "norm")
    ref.close(kept.inv_rms, r[..., 0], r[..., 0].abs() * (ref.chain(x.shape[-1]) / 2 + 5) * ref.u, "inverse rms")
    check_codes(x, kept.x)
    want, tol, dw, dw_tol = ref.norm_backward(x, weight, eps, dy)
    ref.close(grad, want, tol, "norm's gradient")
    if weight is None:
        assert grad_weight is None
    else:
        assert grad_weight.dtype == weight.dtype
        ref.close(grad_weight, dw, dw_tol, "weight's gradient")
    assert same(A.rms_norm(x, weight, eps=eps), y)
    again = A.rms_norm_backward(kept, dy)
    assert same(again[0], grad) and (weight is None or same(again[1], grad_weight))
    return y, kept, grad, grad_weight


NORMS = [(1, 1), (1, 32), (3, 33), (2, 64), (5, 100), (700, 128), (33, 768), (130, 257), (64, 1024), (19, 4096), (2500, 264),
         (3, 5003), (4, 8192), (2, 16384), (3, 40000), (1, 70001), (1, 131072)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,w", NORMS)
def test_norm(n, w, dtype):
    x = make((n, w), dtype, seed=w)
    weight = 1 + make((w,), F32, seed=w + 2, scale=0.1)
    check_norm(x, weight.to(dtype), make((n, w), dtype, seed=w + 1, scale=0.1))


@pytest.mark.parametrize("wtype", [None, BF, F16, F32])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n,w", [(70, 96), (9, 1000), (3, 4104)])
def test_norm_weights(n, w, dtype, wtype):
    x = make((n, w), dtype, seed=w)
    weight = None if wtype is None else (1 + make((w,), F32, seed=w + 2, scale=0.1)).to(wtype)
    check_norm(x, weight, make((n, w), dtype, seed=w + 1, scale=0.1))


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("cut,pad,w", [(0, 8, 96), (1, 0, 96), (3, 5, 100), (4, 12, 52), (0, 1, 768), (8, 8, 4096), (1, 0, 4096)])
def test_norm_of_rows_anywhere(cut, pad, w, dtype):
    n = 21
    x, dy = make((n, w), dtype, seed=w), make((n, w), dtype, seed=w + 1, scale=0.1)
    weight = placed((1 + make((1, w), F32, seed=2, scale=0.1)).to(dtype), cut, 0)[0]
    _, kept, grad, gw = check_norm(placed(x, cut, pad), weight, placed(dy, cut, pad))
    assert torch.equal(A.expand(kept.x), ref.kept(x).float().to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_extremes(dtype):
    w = 300
    x = make((9, w), dtype)
    x[0] = 0.0
    x[1] *= 1e-20
    x[2] *= 1e30                                                 # squares beyond FP32
    x[3] = torch.finfo(dtype).max
    x[4, 7] = INF
    x[5, 299] = NAN
    x[6] *= 1e-38
    weight = (1 + make((w,), F32, seed=3, scale=0.1)).to(dtype)
    y, kept, grad, gw = check_norm(x[:4], weight, make((4, w), dtype, seed=1, scale=0.1), eps=1e-5)
    assert (y[0] == 0).all()
    check_norm(x[:7], weight, make((7, w), dtype, seed=1, scale=0.1), eps=1e-5)   # NaN rows: NaN in the weight's gradient
    check_norm(x[6:], weight, make((3, w), dtype, seed=1, scale=0.1), eps=2.0 ** -80)
    check_norm(x[6:], weight, make((3, w), dtype, seed=1, scale=0.1), eps=2.0 ** 20)


def test_norm_of_no_rows():
    weight = torch.ones(64, dtype=BF, device="cuda")
    y, kept = A.rms_norm_forward(torch.empty(0, 64, dtype=BF, device="cuda"), weight)
    grad, gw = A.rms_norm_backward(kept, y)
    assert grad.shape == (0, 64) and torch.equal(gw, torch.zeros_like(weight))


def test_norm_of_the_longest_rows():
    """More columns than a grid has places in its second dimension times a CTA's threads."""
    w = 20_000_011
    x, dy = torch.zeros(2, w, dtype=BF, device="cuda"), torch.zeros(2, w, dtype=BF, device="cuda")
    at = torch.tensor([0, 1, 16_777_215, 16_777_217, w - 1], device="cuda")
    x[:, at] = make((2, 5), BF) + 3
    dy[:, at] = make((2, 5), BF, seed=1)
    weight = torch.ones(w, dtype=BF, device="cuda")
    y, kept = A.rms_norm_forward(x, weight)
    grad, gw = A.rms_norm_backward(kept, dy)
    r = ref.inverse_rms(x, 1e-6)
    ref.close(y[:, at], (x.double() * r)[:, at], 1e-5, "norm")
    h = (ref.kept(x) * r)[:, at]
    ref.close(gw[at], (dy[:, at].double() * h).sum(0), 1e-4 * (dy[:, at].double() * h).abs().sum(0), "weight's gradient")
    assert int((gw != 0).sum()) == 5
    mean = (dy[:, at].double() * h).sum(1, keepdim=True) / w
    ref.close(grad[:, at], r * (dy[:, at].double() - h * mean), 1e-4 * r, "gradient")


def test_norm_of_many_rows():
    n, w = 300000, 40
    x, weight = make((n, w), BF), torch.ones(w, device="cuda")
    check_norm(x, weight, make((n, w), BF, seed=1, scale=0.1))
