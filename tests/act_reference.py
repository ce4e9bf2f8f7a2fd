"""The operators on activations in 64 bits, from their definitions, and the
tolerances of the tests that compare the kernels with them.

Tolerances (u = 2^-24; U half a step of the result's type). Codes and steps are
exact: their definition fixes every rounding. What is computed from them:
  e^-t        2^-22 from the hardware's exponential; 16-bit types round t at its own
              size: |t| u more, twice for u^2 / 2. FP32 takes t in two parts: 2 u.
  reciprocal  2^-23 (16-bit), 2 u (FP32)
  silu        e and the reciprocal, 1 + e, two products: 2^-22 + 2^-23 + 4 u (16-bit:
              + |x| u), taken as 2^-21 + |x| 2^-23
  gelu        the tail's polynomial: 3.7e-7 < 2^-21 for FP32, 2.2e-6 < 2^-18.7 for
              16-bit types; with e and products 2^-20 or 2^-18, + (x^2 / 2) 2^-22
  slopes      the same relative errors of each of their terms, and a rounding of the sum
  inverse rms a chain of width / 128 + 32 additions of squares at most, halved by the root
  a row's dot product, a column's sum: their number of additions in a chain, of the terms' sizes
and one rounding to the type at the end.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -118, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -118}
u = 2.0 ** -24


def codes(x: torch.Tensor):
    """codes (as float64, [..., 32 G]), steps (float64, [..., G]) of x [..., width], by the definition."""
    width = x.shape[-1]
    g = -(-width // 32)
    y = torch.zeros(x.shape[:-1] + (g * 32,), dtype=torch.float64, device=x.device)
    y[..., :width] = x.double()
    y = y.view(x.shape[:-1] + (g, 32))
    a = y.abs().amax(-1)
    bad = ~torch.isfinite(a)
    want = (torch.where(bad, torch.ones_like(a), a) / 127).clamp(min=2.0 ** -126)
    m, e = torch.frexp(want)
    step = torch.ldexp(torch.ceil(m * 256) / 256, e).float().double()   # a power of two may come out a rounding off
    r = (1 / step).float().double()
    code = torch.round(y * r[..., None])
    step = torch.where(bad, torch.full_like(step, math.nan), step)
    return code.flatten(-2), step


def kept(x: torch.Tensor) -> torch.Tensor:
    """x^ in 64 bits."""
    code, step = codes(x)
    z = code.view(step.shape + (32,)) * step[..., None]
    z = torch.where(torch.isnan(step)[..., None], torch.full_like(z, math.nan), z)
    return z.flatten(-2)[..., :x.shape[-1]]


def act(kind: str, x: torch.Tensor, dtype=None):
    """value, slope, the size of the slope's terms and their relative error for inputs of a type, in 64 bits."""
    dtype = dtype or x.dtype
    x = x.double()
    if kind in ("silu", "swiglu"):
        s, rest = torch.sigmoid(x), torch.sigmoid(-x)
        value = torch.where(x == -math.inf, torch.zeros_like(x), x * s)
        slope, size = s * (1 + x * rest), s * (1 + x.abs() * rest)
        rel = 2.0 ** -21 + x.abs() * 2.0 ** -23
    else:
        cdf = 0.5 * torch.erfc(-x / math.sqrt(2))
        pdf = torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        value = torch.where(x == -math.inf, torch.zeros_like(x), x * cdf)
        slope, size = cdf + x * pdf, cdf + x.abs() * pdf
        rel = (2.0 ** -20 if dtype == torch.float32 else 2.0 ** -18) + x * x * 2.0 ** -23
    return value, slope, size, torch.where(torch.isfinite(rel), rel, torch.zeros_like(rel)).clamp(max=1.0)


def forward(kind, x, up=None):
    """y and its tolerance before the rounding to the type."""
    v, _, _, rel = act(kind, x)
    if up is None:
        return v, v.abs() * rel
    y = v * up.double()
    return y, y.abs() * (rel + u)


def backward(kind, x, dy, up=None):
    """grad, grad_up and their tolerances, at the numbers that the codes of x and up stand for."""
    xh, dy = kept(x), dy.double()
    v, slope, size, rel = act(kind, xh, x.dtype)
    if up is None:
        return dy * slope, dy.abs() * size * (rel + 2 * u)
    uh = kept(up)
    return (dy * uh * slope, (dy * uh).abs() * size * (rel + 3 * u), dy * v, (dy * v).abs() * (rel + u))


def inverse_rms(x, eps):
    s = x.double()
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return torch.where(torch.isfinite(s).all(-1, keepdim=True), r, torch.full_like(r, math.nan))


def chain(width: int) -> float:
    return width / 128 + 32


def norm(x, weight, eps):
    r = inverse_rms(x, eps)
    y = x.double() * r * (1 if weight is None else weight.double())
    return y, y.abs() * (chain(x.shape[-1]) / 2 + 5) * u, r


def norm_backward(x, weight, eps, dy):
    """grad, its tolerance, grad_weight, its tolerance. x [rows, width]."""
    r, dy = inverse_rms(x, eps), dy.double()
    h = kept(x) * r
    g = dy * (1 if weight is None else weight.double())
    width, rows = x.shape[-1], x.shape[0]
    mean, size = (g * h).mean(-1, keepdim=True), (g * h).abs().mean(-1, keepdim=True)
    grad = r * (g - h * mean)
    a = (chain(width) / 2 + 5) * u                       # of r
    tol = r * (g.abs() * (a + 3 * u) + h.abs() * size * (3 * a + (chain(width) + 6) * u))
    dw, dw_size = (dy * h).sum(0), (dy * h).abs().sum(0)
    additions = rows / min(max(rows, 1), 1024) + 1024 / 8 + 32
    return grad, tol, dw, dw_size * (a + additions * u)


def close(got, want, tol, what):
    """Equal where `want`, as a value of the result's type, is not finite (either side may
    round up to infinity within the tolerance); within one rounding and tol elsewhere."""
    dt = got.dtype
    limit = torch.finfo(dt).max
    got, want = got.double(), want.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(want.shape)}"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    tol = torch.nan_to_num(torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand_as(want), nan=0.0)
    over = torch.isfinite(want) & (want.abs() + tol >= limit * (1 - 2.0 ** -12))    # may round to infinity
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    assert torch.equal(torch.sign(got[over]), torch.sign(want[over])), f"{what}: largest values differ"
    fine = torch.isfinite(want) & ~over
    assert torch.isfinite(got[fine]).all(), f"{what}: not finite where it should be"
    allowed = tol * (1 + UNIT[dt]) + UNIT[dt] * want.abs() * (1 + 2.0 ** -9) + TINY[dt]
    off = ((got - want).abs() - allowed)[fine]
    if off.numel():
        i = int(off.argmax())
        assert float(off[i]) <= 0, (f"{what}: off by {float((got - want).abs()[fine][i]):.3g}, allowed "
                                    f"{float(allowed[fine][i]):.3g}, at value {float(want[fine][i]):.6g}")
