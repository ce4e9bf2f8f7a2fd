"""Activations kept for the backward pass in 8 bits, through the library's
kernels: beside the optimizer state, what a training step holds in memory.

* :func:`compress`, :func:`expand` -- a tensor to int8 codes with one bfloat16
  step for every 32 elements of its last dimension, and back;
* :func:`activation` -- ``silu``, ``gelu``, and the gated ``swiglu`` and ``geglu``;
* :func:`rms_norm` -- root-mean-square norm;
* :func:`linear` -- a matrix product whose input is kept the same way.

The last three are differentiable. Their results are those of the input itself;
what they keep of it for the backward pass are its codes (1.0625 bytes an element
where bfloat16 takes 2), and the gradient is the formula's at the numbers that
the codes stand for, within half a step (1/254 of a group's largest) of the input.
Training loops that run the backward pass themselves have the calls in pairs:
:func:`activation_forward` and :func:`activation_backward`, :func:`rms_norm_forward`
and :func:`rms_norm_backward`.

Tensors are bfloat16, float16 or float32 on the current CUDA device, ``[..., width]``
with a contiguous last dimension and the rows one stride apart: ``x[:, :k]`` is
read where it lies. The code, and the rules for infinities and NaN, stand in
``include/fo.h``. Work is enqueued on the current stream. Derivatives are of the
first order and in reverse mode; a tangent of forward mode is refused.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import fo
from .losses import _on_device_of

KINDS = {"silu": (fo.FO_ACT_SILU, False), "gelu": (fo.FO_ACT_GELU, False),
         "swiglu": (fo.FO_ACT_SILU, True), "geglu": (fo.FO_ACT_GELU, True)}


class Compressed(NamedTuple):
    """A tensor in 8 bits: an element is ``codes * steps`` of its group."""
    codes: torch.Tensor      # [..., 32 G] int8, G = ceil(width / 32)
    steps: torch.Tensor      # [..., G] bfloat16
    width: int
    dtype: torch.dtype


class KeptActivation(NamedTuple):
    """What :func:`activation_backward` needs."""
    kind: str
    codes: torch.Tensor      # [..., 32 G] int8; [2, ..., 32 G] of a gated kind: the gate's and the other half's
    steps: torch.Tensor      # [..., G] or [2, ..., G] bfloat16
    shape: torch.Size        # of the result
    dtype: torch.dtype
    halves: bool             # gate and other half are those of one tensor


class KeptNorm(NamedTuple):
    """What :func:`rms_norm_backward` needs. ``weight`` is the tensor itself, not a copy."""
    x: Compressed
    inv_rms: torch.Tensor    # [...] float32
    weight: Optional[torch.Tensor]


def _check_tangent(*tensors: Optional[torch.Tensor]) -> None:
    """A tensor with a tangent need not require a gradient, and its address carries none."""
    for x in tensors:
        if x is not None and forward_ad.unpack_dual(x).tangent is not None:
            raise NotImplementedError("operators on activations have no forward-mode derivative: an input carries a tangent")


def _check_width(x: torch.Tensor) -> None:
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"a tensor [..., width] of at least one column is needed, not {tuple(x.shape)}")


# The functions below hand the C calls the addresses of tensors that they have
# just made themselves; what the caller passes is checked by fo's helpers.

def _empty_kept(lead, width: int, device):
    g = fo.groups(width)
    return (torch.empty(lead + (g * fo.GROUP,), dtype=torch.int8, device=device),
            torch.empty(lead + (g,), dtype=torch.bfloat16, device=device))


def _grad_of(grad: torch.Tensor, shape, dtype, name: str = "grad_y") -> torch.Tensor:
    """An incoming gradient in a layout that the kernels read (an expanded one, for example, is copied)."""
    if grad.shape != shape or grad.dtype != dtype:
        raise ValueError(f"{name} must be {str(dtype).replace('torch.', '')} of shape {tuple(shape)}, not "
                         f"{str(grad.dtype).replace('torch.', '')} of shape {tuple(grad.shape)}")
    return grad if fo._rows_of(grad) is not None else grad.contiguous()


def compress(x: torch.Tensor) -> Compressed:
    """The codes and steps of ``x``; groups of 32 run along the last dimension, the
    last one of a row may be partial. Not differentiable."""
    _check_tangent(x)
    _check_width(x)
    m = fo.matrix(x)
    codes, steps = _empty_kept(x.shape[:-1], x.shape[-1], x.device)
    status = fo.lib().fo_compress(ctypes.byref(m), codes.data_ptr(), steps.data_ptr(), fo._stream(None))
    if status:
        fo._check("fo_compress", status)
    return Compressed(codes, steps, x.shape[-1], x.dtype)


def expand(kept: Compressed, *, dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The tensor that the codes stand for, rounded once to ``dtype`` (that of the
    compressed tensor where None). ``out``: where to write it."""
    codes, steps, width, own = kept
    lead = codes.shape[:-1]
    if steps.shape != lead + (fo.groups(width),) or codes.shape[-1] != fo.groups(width) * fo.GROUP:
        raise ValueError(f"codes {tuple(codes.shape)} and steps {tuple(steps.shape)} are not those of {width} columns")
    if out is None:
        x = torch.empty(lead + (width,), dtype=dtype or own, device=codes.device)
    elif out.shape != lead + (width,) or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must be of shape {tuple(lead + (width,))}" + (f" and {dtype}" if dtype else "") +
                         f", not {tuple(out.shape)} and {out.dtype}")
    else:
        x = out
    fo.fo_expand(codes, steps, x)
    return x


# --- activation functions ------------------------------------------------------------------

def _activation(x, kind, up, keep):
    try:
        act, gated = KINDS[kind]
    except (KeyError, TypeError):
        raise ValueError(f"kind must be one of {', '.join(KINDS)}, not {kind!r}") from None
    _check_width(x)
    if up is not None and not gated:
        raise ValueError(f"{kind} takes no second input")
    halves = gated and up is None
    m, u = fo.matrix(x), None
    shape = x.shape
    if halves:
        if shape[-1] % 2:
            raise ValueError(f"{kind} halves the last dimension, which must be even, not {shape[-1]}")
        shape = shape[:-1] + (shape[-1] // 2,)
        m.width = shape[-1]
        u = fo.FoRows(m.data + m.width * x.element_size(), m.rows, m.width, m.row_stride, m.dtype, 0)
    elif gated:
        if up.shape != shape:
            raise ValueError(f"up must have the gate's shape {tuple(shape)}, not {tuple(up.shape)}")
        u = fo.matrix(up, "up", m)
    y = torch.empty(shape, dtype=x.dtype, device=x.device)
    width = shape[-1]
    to = fo.FoRows(y.data_ptr(), m.rows, width, width, m.dtype, 0)
    codes = steps = c = s = uc = us = None
    if keep:
        codes, steps = _empty_kept(((2,) if gated else ()) + shape[:-1], width, x.device)
        c, s = codes.data_ptr(), steps.data_ptr()
        if gated:
            half = m.rows * fo.groups(width)
            uc, us = c + half * fo.GROUP, s + half * 2
    status = fo.lib().fo_activation(act, ctypes.byref(m), fo._ref(u), ctypes.byref(to), c, s, uc, us, fo._stream(None))
    if status:
        fo._check("fo_activation", status)
    return y, KeptActivation(kind, codes, steps, shape, x.dtype, halves) if keep else None


def activation_forward(x: torch.Tensor, kind: str, *, up: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, KeptActivation]:
    """``(y, kept)``: :func:`activation` and what :func:`activation_backward` needs."""
    _check_tangent(x, up)
    return _activation(x, kind, up, True)


def activation_backward(kept: KeptActivation, grad_y: torch.Tensor):
    """The gradient of ``x`` (of ``(x, up)`` where ``up`` was given) for that of ``y``."""
    kind, codes, steps, shape, dtype, halves = kept
    act, gated = KINDS[kind]
    grad_y = _grad_of(grad_y, shape, dtype)
    m = fo.matrix(grad_y, "grad_y")
    width, size = m.width, grad_y.element_size()
    cur = grad_y.device.index
    n = m.rows * fo.groups(width) * (2 if gated else 1)
    c = fo._array(codes, "codes", torch.int8, n * fo.GROUP, cur)
    s = fo._array(steps, "steps", torch.bfloat16, n, cur)
    grad_up = to_up = uc = us = None
    stride = 2 * width if halves else width
    grad = torch.empty(shape[:-1] + (stride,), dtype=dtype, device=grad_y.device)
    to = fo.FoRows(grad.data_ptr(), m.rows, width, stride, m.dtype, 0)
    if gated:
        if halves:
            at = to.data + width * size if m.rows else None
        else:
            grad_up = torch.empty_like(grad)
            at = grad_up.data_ptr()
        to_up = fo.FoRows(at, m.rows, width, stride, m.dtype, 0)
        if m.rows:
            uc, us = c + n // 2 * fo.GROUP, s + n // 2 * 2
    status = fo.lib().fo_activation_grad(act, c, s, uc, us, ctypes.byref(m), ctypes.byref(to), fo._ref(to_up), fo._stream(None))
    if status:
        fo._check("fo_activation_grad", status)
    return (grad, grad_up) if gated and not halves else grad


class _Activation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, up, kind):
        y, kept = _activation(x, kind, up, True)
        ctx.save_for_backward(kept.codes, kept.steps)
        ctx.how = (kept.shape, kept.dtype, kept.halves)
        ctx.kind = kind
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        codes, steps = ctx.saved_tensors
        with _on_device_of(codes):
            grad = activation_backward(KeptActivation(ctx.kind, codes, steps, *ctx.how), grad_y)
        return (*grad, None) if isinstance(grad, tuple) else (grad, None, None)


def _differentiable(*tensors) -> bool:
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def activation(x: torch.Tensor, kind: str, *, up: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``silu(x)``, ``gelu(x)`` (exact, not its tanh form), or of the gated kinds
    ``silu(gate) * up`` (``swiglu``) and ``gelu(gate) * up`` (``geglu``), whose gate and
    ``up`` are the halves of ``x`` along the last dimension, or ``x`` and ``up``.
    Differentiable; the input is kept in 8 bits where a gradient is asked for."""
    _check_tangent(x, up)
    if _differentiable(x, up):
        return _Activation.apply(x, up, kind)
    return _activation(x, kind, up, False)[0]


# --- norm ------------------------------------------------------------------------------------

def _norm(x, weight, eps, keep):
    _check_width(x)
    m, width, dev = fo.matrix(x), x.shape[-1], x.device
    w, wt = None, 0
    if weight is not None:
        if weight.shape != (width,):
            raise ValueError(f"weight must be of shape ({width},), not {tuple(weight.shape)}")
        w, wt = fo._weight(weight, "weight", width, dev.index)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    to = fo.FoRows(y.data_ptr(), m.rows, width, width, m.dtype, 0)
    codes = steps = inv = c = s = p_inv = None
    if keep:
        codes, steps = _empty_kept(x.shape[:-1], width, dev)
        inv = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        c, s, p_inv = codes.data_ptr(), steps.data_ptr(), inv.data_ptr()
    status = fo.lib().fo_rms_norm(ctypes.byref(m), w, wt, eps, ctypes.byref(to), p_inv, c, s, fo._stream(None))
    if status:
        fo._check("fo_rms_norm", status)
    return y, KeptNorm(Compressed(codes, steps, width, x.dtype), inv, weight) if keep else None


def rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> Tuple[torch.Tensor, KeptNorm]:
    """``(y, kept)``: :func:`rms_norm` and what :func:`rms_norm_backward` needs."""
    _check_tangent(x, weight)
    return _norm(x, weight, eps, True)


def _norm_backward(kept, grad_y, need_x, need_weight):
    x, inv, weight = kept
    shape = x.codes.shape[:-1] + (x.width,)
    grad_y = _grad_of(grad_y, shape, x.dtype)
    m, dev, f32 = fo.matrix(grad_y, "grad_y"), grad_y.device, torch.float32
    cur = dev.index
    c, s = fo._kept(x.codes, x.steps, m, cur)
    w, wt = fo._weight(weight, "weight", m.width, cur)
    grad = to = grad_weight = gw = parts = ws = None
    if need_x:
        grad = torch.empty(shape, dtype=x.dtype, device=dev)
        to = fo.FoRows(grad.data_ptr(), m.rows, m.width, m.width, m.dtype, 0)
    if need_weight and weight is not None:
        grad_weight = torch.empty_like(weight)
        parts = torch.empty(min(m.rows, fo.FO_NORM_PARTS) * fo.groups(m.width) * fo.GROUP, dtype=f32, device=dev)
        gw, ws = grad_weight.data_ptr(), parts.data_ptr()
    status = fo.lib().fo_rms_norm_grad(c, s, fo._array(inv, "inv_rms", f32, m.rows, cur), w, wt, ctypes.byref(m), fo._ref(to),
                                       gw, ws, fo._stream(None))
    if status:
        fo._check("fo_rms_norm_grad", status)
    return grad, grad_weight


def rms_norm_backward(kept: KeptNorm, grad_y: torch.Tensor) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``(grad_x, grad_weight)`` for the gradient of ``y``; ``grad_weight``, of the
    weight's type, is None without one."""
    return _norm_backward(kept, grad_y, True, True)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps):
        y, kept = _norm(x, weight, eps, True)
        ctx.save_for_backward(kept.x.codes, kept.x.steps, kept.inv_rms, weight)
        ctx.how = (kept.x.width, kept.x.dtype)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        codes, steps, inv, weight = ctx.saved_tensors
        with _on_device_of(codes):
            kept = KeptNorm(Compressed(codes, steps, *ctx.how), inv, weight)
            return (*_norm_backward(kept, grad_y, ctx.needs_input_grad[0], ctx.needs_input_grad[1]), None)


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> torch.Tensor:
    """``x / sqrt(mean(x^2) + eps) * weight`` over the last dimension, in ``x``'s type;
    ``weight`` [width] may be of another one. ``eps`` in [2^-80, 2^20].
    Differentiable; ``x`` is kept in 8 bits where a gradient is asked for. The
    gradient of ``weight`` sums the rows in FP32, in an order that depends on
    their number only."""
    _check_tangent(x, weight)
    if _differentiable(x, weight):
        return _Norm.apply(x, weight, eps)
    return _norm(x, weight, eps, False)[0]


# --- matrix product ---------------------------------------------------------------------------

class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        kept = compress(x) if ctx.needs_input_grad[1] else None
        ctx.save_for_backward(weight, *(kept[:2] if kept else ()))
        ctx.how = (x.shape[-1], x.dtype)
        with torch.autocast("cuda", enabled=False):
            return torch.nn.functional.linear(x, weight, bias)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        weight, *kept = ctx.saved_tensors
        grad_x = grad_weight = grad_bias = None
        with _on_device_of(weight), torch.autocast("cuda", enabled=False):
            rows = grad_y.reshape(-1, grad_y.shape[-1])
            if ctx.needs_input_grad[0]:
                grad_x = grad_y @ weight
            if ctx.needs_input_grad[1]:
                x = expand(Compressed(*kept, *ctx.how))
                grad_weight = rows.t() @ x.view(-1, x.shape[-1])
            if ctx.needs_input_grad[2]:
                grad_bias = rows.sum(0)
        return grad_x, grad_weight, grad_bias


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``x @ weight.t() + bias`` with ``x`` kept in 8 bits for the gradient of
    ``weight``, which is a matrix product with the expanded copy (that of ``x``
    needs the weight alone). One type for all."""
    _check_tangent(x, weight, bias)
    if x.dtype != weight.dtype or (bias is not None and bias.dtype != x.dtype):
        raise TypeError(f"x, weight and bias must be of one type, not {x.dtype}, {weight.dtype}" +
                        (f" and {bias.dtype}" if bias is not None else ""))
    if _differentiable(x, weight, bias):
        return _Linear.apply(x, weight, bias)
    return torch.nn.functional.linear(x, weight, bias)
