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
    kept: torch.Tensor       # bytes: codes of the input (of a gated kind the gate's, then the other half's), then steps
    shape: torch.Size        # of the result
    dtype: torch.dtype
    halves: bool             # gate and other half are those of one tensor

    def inputs(self) -> Tuple[Compressed, ...]:
        """The input, or the gate and the other half."""
        n, width = self.shape[:-1].numel(), self.shape[-1]
        g, parts = fo.groups(width), 2 if KINDS[self.kind][1] else 1
        codes = self.kept[:parts * n * g * fo.GROUP].view((parts,) + self.shape[:-1] + (g * fo.GROUP,))
        steps = self.kept[parts * n * g * fo.GROUP:].view(torch.bfloat16).view((parts,) + self.shape[:-1] + (g,))
        return tuple(Compressed(c, s, width, self.dtype) for c, s in zip(codes, steps))


class KeptNorm(NamedTuple):
    """What :func:`rms_norm_backward` needs. ``weight`` is the tensor itself, not a copy."""
    kept: torch.Tensor       # bytes: codes of the input, then 1 / rms of each row, then steps
    shape: torch.Size
    dtype: torch.dtype
    weight: Optional[torch.Tensor]

    @property
    def x(self) -> Compressed:
        """The input."""
        n, g = self.shape[:-1].numel(), fo.groups(self.shape[-1])
        codes = self.kept[:n * g * fo.GROUP].view(self.shape[:-1] + (g * fo.GROUP,))
        steps = self.kept[n * (g * fo.GROUP + 4):].view(torch.bfloat16).view(self.shape[:-1] + (g,))
        return Compressed(codes, steps, self.shape[-1], self.dtype)

    @property
    def inv_rms(self) -> torch.Tensor:
        """1 / rms of each row, float32."""
        at = self.shape[:-1].numel() * fo.groups(self.shape[-1]) * fo.GROUP
        return self.kept[at:at + 4 * self.shape[:-1].numel()].view(torch.float32).view(self.shape[:-1])


def _check_tangent(*tensors: Optional[torch.Tensor]) -> None:
    """A tensor with a tangent need not require a gradient, and its address carries none."""
    if getattr(forward_ad, "_current_level", 0) < 0:     # outside of every forward-mode level there are none
        return
    for x in tensors:
        if x is not None and forward_ad.unpack_dual(x).tangent is not None:
            raise NotImplementedError("operators on activations have no forward-mode derivative: an input carries a tangent")


def _check_width(x: torch.Tensor) -> None:
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"a tensor [..., width] of at least one column is needed, not {tuple(x.shape)}")


# The functions below hand the C calls the addresses of tensors that they have
# just made themselves; what the caller passes is checked by fo's helpers. A call
# is a few microseconds of host time, which is what small tensors take.

_empty = torch.empty


def _grad_rows(grad: torch.Tensor, shape, dtype, rows: int, dt: int) -> fo.FoRows:
    """An incoming gradient of the result's shape and type (``rows`` and ``dt`` are theirs). One in a
    layout that the kernels do not read (an expanded one, for example) is copied; the rows hold the copy."""
    if grad.dtype is dtype and grad.shape == shape and grad.is_contiguous() and grad.get_device() == fo._current_device():
        width = shape[-1]
        return fo.FoRows(grad.data_ptr(), rows, width, width, dt, 0)
    if grad.shape != shape or grad.dtype != dtype:
        raise ValueError(f"grad_y must be {str(dtype).replace('torch.', '')} of shape {tuple(shape)}, not "
                         f"{str(grad.dtype).replace('torch.', '')} of shape {tuple(grad.shape)}")
    if fo._rows_of(grad) is None:
        grad = grad.contiguous()
    m = fo.matrix(grad, "grad_y")
    m.keep = grad
    return m


def compress(x: torch.Tensor) -> Compressed:
    """The codes and steps of ``x``; groups of 32 run along the last dimension, the
    last one of a row may be partial. Not differentiable."""
    _check_tangent(x)
    _check_width(x)
    m = fo.matrix(x)
    shape, dev = x.shape, x.device
    g = -(-m.width // fo.GROUP)
    lead = shape[:-1]
    codes = _empty(lead + (g * fo.GROUP,), dtype=torch.int8, device=dev)
    steps = _empty(lead + (g,), dtype=torch.bfloat16, device=dev)
    status = fo.lib().fo_compress(ctypes.byref(m), codes.data_ptr(), steps.data_ptr(), fo._stream(None))
    if status:
        fo._check("fo_compress", status)
    return Compressed(codes, steps, m.width, x.dtype)


def expand(kept: Compressed, *, dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The tensor that the codes stand for, rounded once to ``dtype`` (that of the
    compressed tensor where None). ``out``: where to write it."""
    codes, steps, width, own = kept
    lead, g = codes.shape[:-1], -(-width // fo.GROUP)
    if steps.shape != lead + (g,) or codes.shape[-1] != g * fo.GROUP:
        raise ValueError(f"codes {tuple(codes.shape)} and steps {tuple(steps.shape)} are not those of {width} columns")
    if out is not None:
        if out.shape != lead + (width,) or (dtype is not None and out.dtype != dtype):
            raise ValueError(f"out must be of shape {tuple(lead + (width,))}" + (f" and {dtype}" if dtype else "") +
                             f", not {tuple(out.shape)} and {out.dtype}")
        fo.fo_expand(codes, steps, out)
        return out
    x = _empty(lead + (width,), dtype=dtype or own, device=codes.device)
    m = fo.matrix(x)
    c, s = fo._kept(codes, steps, m, x.device.index)
    status = fo.lib().fo_expand(c, s, ctypes.byref(m), fo._stream(None))
    if status:
        fo._check("fo_expand", status)
    return x


# --- activation functions ------------------------------------------------------------------

def _activation(x, kind, up, keep):
    """(the result, the bytes that are kept or None, what :func:`_activation_grad` needs beside them)"""
    try:
        act, gated = KINDS[kind]
    except (KeyError, TypeError):
        raise ValueError(f"kind must be one of {', '.join(KINDS)}, not {kind!r}") from None
    _check_width(x)
    if up is not None and not gated:
        raise ValueError(f"{kind} takes no second input")
    m, u, shape, dtype, dev = fo.matrix(x), None, x.shape, x.dtype, x.device
    width, rows, dt = m.width, m.rows, m.dtype
    if gated:
        if up is None:
            if width % 2:
                raise ValueError(f"{kind} halves the last dimension, which must be even, not {width}")
            width //= 2
            shape = shape[:-1] + (width,)
            m.width = width
            u = ctypes.byref(fo.FoRows((m.data or 0) + width * x.element_size(), rows, width, m.row_stride, dt, 0))
        else:
            if up.shape != shape:
                raise ValueError(f"up must have the gate's shape {tuple(shape)}, not {tuple(up.shape)}")
            u = ctypes.byref(fo.matrix(up, "up", m))
    y = _empty(shape, dtype=dtype, device=dev)
    kept = c = s = uc = us = None
    if keep:
        n = rows * -(-width // fo.GROUP)          # groups
        kept = _empty(n * (68 if gated else 34), dtype=torch.int8, device=dev)
        c = kept.data_ptr()
        s = c + n * fo.GROUP
        if gated:
            uc, s = s, s + n * fo.GROUP
            us = s + 2 * n
    status = fo.lib().fo_activation(act, ctypes.byref(m), u, ctypes.byref(fo.FoRows(y.data_ptr(), rows, width, width, dt, 0)),
                                    c, s, uc, us, fo._stream(None))
    if status:
        fo._check("fo_activation", status)
    return y, kept, (act, gated, gated and up is None, shape, dtype, rows, dt)


def _activation_grad(kept, how, grad_y):
    act, gated, halves, shape, dtype, rows, dt = how
    m = _grad_rows(grad_y, shape, dtype, rows, dt)
    width, dev = shape[-1], kept.device
    n = rows * -(-width // fo.GROUP)
    c = kept.data_ptr()
    s = c + n * fo.GROUP
    grad_up = uc = us = to_up = None
    if halves:
        stride = 2 * width
        grad = _empty(shape[:-1] + (stride,), dtype=dtype, device=dev)
    else:
        stride = width
        grad = _empty(shape, dtype=dtype, device=dev)
    at = grad.data_ptr()
    if gated:
        uc, s = s, s + n * fo.GROUP
        us = s + 2 * n
        if not halves:
            grad_up = torch.empty_like(grad)
        to_up = ctypes.byref(fo.FoRows(at + width * grad.element_size() if halves else grad_up.data_ptr(), rows, width, stride, dt, 0))
    status = fo.lib().fo_activation_grad(act, c, s, uc, us, ctypes.byref(m), ctypes.byref(fo.FoRows(at, rows, width, stride, dt, 0)),
                                         to_up, fo._stream(None))
    if status:
        fo._check("fo_activation_grad", status)
    return grad, grad_up


def activation_forward(x: torch.Tensor, kind: str, *, up: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, KeptActivation]:
    """``(y, kept)``: :func:`activation` and what :func:`activation_backward` needs."""
    _check_tangent(x, up)
    y, kept, how = _activation(x, kind, up, True)
    return y, KeptActivation(kind, kept, y.shape, y.dtype, how[2])


def activation_backward(kept: KeptActivation, grad_y: torch.Tensor):
    """The gradient of ``x`` (of ``(x, up)`` where ``up`` was given) for that of ``y``."""
    kind, buffer, shape, dtype, halves = kept
    act, gated = KINDS[kind]
    rows = shape[:-1].numel()
    fo._array(buffer, "kept", torch.int8, rows * -(-shape[-1] // fo.GROUP) * (68 if gated else 34), fo._current_device())
    grad, grad_up = _activation_grad(buffer, (act, gated, halves, shape, dtype, rows, fo._logit_dtype(dtype, "kept")), grad_y)
    return grad if grad_up is None else (grad, grad_up)


class _Activation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, up, kind):
        y, kept, ctx.how = _activation(x, kind, up, True)
        ctx.save_for_backward(kept)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        kept, = ctx.saved_tensors
        if kept.get_device() == fo._current_device():
            return (*_activation_grad(kept, ctx.how, grad_y), None)
        with torch.cuda.device(kept.device):
            return (*_activation_grad(kept, ctx.how, grad_y), None)


def _differentiable(*tensors) -> bool:
    return torch.is_grad_enabled() and any([t is not None and t.requires_grad for t in tensors])


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
    """(the result, the bytes that are kept or None, what :func:`_norm_grad` needs beside them)"""
    _check_width(x)
    m, dev, shape = fo.matrix(x), x.device, x.shape
    width, rows = m.width, m.rows
    w, wt = None, 0
    if weight is not None:
        if weight.shape != shape[-1:]:
            raise ValueError(f"weight must be of shape ({width},), not {tuple(weight.shape)}")
        w, wt = fo._weight(weight, "weight", width, dev.index)
    y = _empty(shape, dtype=x.dtype, device=dev)
    kept = c = s = inv = None
    if keep:
        n = rows * -(-width // fo.GROUP)          # groups
        kept = _empty(n * 34 + 4 * rows, dtype=torch.int8, device=dev)
        c = kept.data_ptr()
        inv = c + n * fo.GROUP
        s = inv + 4 * rows
    status = fo.lib().fo_rms_norm(ctypes.byref(m), w, wt, eps, ctypes.byref(fo.FoRows(y.data_ptr(), rows, width, width, m.dtype, 0)),
                                  inv, c, s, fo._stream(None))
    if status:
        fo._check("fo_rms_norm", status)
    return y, kept, (shape, x.dtype, rows, m.dtype, wt)


def _norm_grad(kept, weight, how, grad_y, need_x, need_weight):
    shape, dtype, rows, dt, wt = how
    m = _grad_rows(grad_y, shape, dtype, rows, dt)
    width, dev = shape[-1], kept.device
    c = kept.data_ptr()
    inv = c + rows * -(-width // fo.GROUP) * fo.GROUP
    w = None if weight is None else weight.data_ptr()
    grad = to = grad_weight = gw = parts = ws = None
    if need_x:
        grad = _empty(shape, dtype=dtype, device=dev)
        to = ctypes.byref(fo.FoRows(grad.data_ptr(), rows, width, width, dt, 0))
    if need_weight and weight is not None:
        grad_weight = torch.empty_like(weight)
        parts = _empty(fo.lib().fo_rms_norm_workspace(rows, width), dtype=torch.float32, device=dev)
        gw, ws = grad_weight.data_ptr(), parts.data_ptr()
    status = fo.lib().fo_rms_norm_grad(c, inv + 4 * rows, inv, w, wt, ctypes.byref(m), to, gw, ws, fo._stream(None))
    if status:
        fo._check("fo_rms_norm_grad", status)
    return grad, grad_weight


def rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> Tuple[torch.Tensor, KeptNorm]:
    """``(y, kept)``: :func:`rms_norm` and what :func:`rms_norm_backward` needs."""
    _check_tangent(x, weight)
    y, kept, _ = _norm(x, weight, eps, True)
    return y, KeptNorm(kept, y.shape, y.dtype, weight)


def rms_norm_backward(kept: KeptNorm, grad_y: torch.Tensor) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``(grad_x, grad_weight)`` for the gradient of ``y``; ``grad_weight``, of the
    weight's type, is None without one."""
    buffer, shape, dtype, weight = kept
    rows, cur = shape[:-1].numel(), fo._current_device()
    fo._array(buffer, "kept", torch.int8, rows * (-(-shape[-1] // fo.GROUP) * 34 + 4), cur)
    _, wt = fo._weight(weight, "weight", shape[-1], cur)
    return _norm_grad(buffer, weight, (shape, dtype, rows, fo._logit_dtype(dtype, "kept"), wt), grad_y, True, True)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps):
        y, kept, ctx.how = _norm(x, weight, eps, True)
        ctx.save_for_backward(kept, weight)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y):
        kept, weight = ctx.saved_tensors
        need_x, need_weight, _ = ctx.needs_input_grad
        if kept.get_device() == fo._current_device():
            return (*_norm_grad(kept, weight, ctx.how, grad_y, need_x, need_weight), None)
        with torch.cuda.device(kept.device):
            return (*_norm_grad(kept, weight, ctx.how, grad_y, need_x, need_weight), None)


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> torch.Tensor:
    """``x / sqrt(mean(x^2) + eps) * weight`` over the last dimension, in ``x``'s type;
    ``weight`` [width] may be of another one. ``eps`` in [2^-80, 2^20].
    Differentiable; ``x`` is kept in 8 bits where a gradient is asked for. The
    gradient of ``weight`` sums the rows in FP32, in an order that depends on their
    number and the device only."""
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
