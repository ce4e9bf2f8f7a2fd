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
the codes stand for, within half a step (at most 1/252 of a group's largest, or
2^-127) of the input.
Training loops that run the backward pass themselves have the calls in pairs:
:func:`activation_forward` and :func:`activation_backward`, :func:`rms_norm_forward`
and :func:`rms_norm_backward`.

Tensors are bfloat16, float16 or float32 on the current CUDA device, ``[..., width]``
with a contiguous last dimension and the rows one stride apart: ``x[:, :k]`` is
read where it lies. The code, and the rules for infinities and NaN, stand in
``include/fo.h``. Work is enqueued on the current stream; calls can be captured in
CUDA graphs, their temporaries are the graph's own (a backward pass by
``torch.autograd.grad``, or with no eager graph of the same leaves alive, as PyTorch
asks of every captured one). Derivatives are of the first order and in reverse mode;
a tangent of forward mode is refused.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import fo

_native = fo.native

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


def compress(x: torch.Tensor) -> Compressed:
    """The codes and steps of ``x``; groups of 32 run along the last dimension, the
    last one of a row may be partial. Not differentiable."""
    _check_tangent(x)
    codes, steps = _native().compress(x)
    return Compressed(codes, steps, x.shape[-1], x.dtype)


def expand(kept: Compressed, *, dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The tensor that the codes stand for, rounded once to ``dtype`` (that of the
    compressed tensor where None, in which numbers come back as numbers: next to the
    type's largest a code may stand for more, and gives the largest). ``out``: where to
    write it."""
    codes, steps, width, own = kept
    if out is not None and dtype is not None and out.dtype != dtype:
        raise ValueError(f"out must be {dtype}, not {out.dtype}")
    return _native().expand(codes, steps, width, dtype or own, out)


# --- activation functions ------------------------------------------------------------------

def _kind(kind: str, up: Optional[torch.Tensor]) -> Tuple[int, bool]:
    """(fo_act_t, whether the kind is gated)"""
    try:
        how = KINDS[kind]
    except (KeyError, TypeError):
        raise ValueError(f"kind must be one of {', '.join(KINDS)}, not {kind!r}") from None
    if up is not None and not how[1]:
        raise ValueError(f"{kind} takes no second input")
    return how


def activation(x: torch.Tensor, kind: str, *, up: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``silu(x)``, ``gelu(x)`` (exact, not its tanh form), or of the gated kinds
    ``silu(gate) * up`` (``swiglu``) and ``gelu(gate) * up`` (``geglu``), whose gate and
    ``up`` are the halves of ``x`` along the last dimension, or ``x`` and ``up``.
    Differentiable; the input is kept in 8 bits where a gradient is asked for."""
    _check_tangent(x, up)
    return _native().activation(x, up, *_kind(kind, up))


def activation_forward(x: torch.Tensor, kind: str, *, up: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, KeptActivation]:
    """``(y, kept)``: :func:`activation` and what :func:`activation_backward` needs."""
    _check_tangent(x, up)
    act, gated = _kind(kind, up)
    y, kept = _native().activation_forward(x, up, act, gated)
    return y, KeptActivation(kind, kept, y.shape, y.dtype, gated and up is None)


def activation_backward(kept: KeptActivation, grad_y: torch.Tensor):
    """The gradient of ``x`` (of ``(x, up)`` where ``up`` was given) for that of ``y``."""
    _check_tangent(grad_y)
    kind, buffer, shape, dtype, halves = kept
    act, gated = KINDS[kind]
    grads = _native().activation_backward(buffer, act, gated, halves, shape, dtype, grad_y)
    return grads if gated and not halves else grads[0]


# --- norm ------------------------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> torch.Tensor:
    """``x / sqrt(mean(x^2) + eps) * weight`` over the last dimension, in ``x``'s type;
    ``weight`` [width] may be of another one. ``eps`` in [2^-80, 2^20].
    Differentiable; ``x`` is kept in 8 bits where a gradient is asked for. The
    gradient of ``weight`` sums the rows in FP32 (a 152th of them or fewer one after
    another), in an order that depends on their number and the device only."""
    _check_tangent(x, weight)
    return _native().rms_norm(x, weight, eps)


def rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6) -> Tuple[torch.Tensor, KeptNorm]:
    """``(y, kept)``: :func:`rms_norm` and what :func:`rms_norm_backward` needs."""
    _check_tangent(x, weight)
    y, kept = _native().rms_norm_forward(x, weight, eps)
    return y, KeptNorm(kept, y.shape, y.dtype, weight)


def rms_norm_backward(kept: KeptNorm, grad_y: torch.Tensor) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``(grad_x, grad_weight)`` for the gradient of ``y``; ``grad_weight``, of the
    weight's type, is None without one."""
    buffer, shape, dtype, weight = kept
    _check_tangent(grad_y, weight)
    return _native().rms_norm_backward(buffer, shape, dtype, weight, grad_y)


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
    def backward(ctx, grad_y):
        weight, *kept = ctx.saved_tensors
        grad_x = grad_weight = grad_bias = None
        with torch.cuda.device(weight.device), torch.autocast("cuda", enabled=False), torch.no_grad():
            rows = grad_y.reshape(-1, grad_y.shape[-1])
            if ctx.needs_input_grad[0]:
                grad_x = grad_y @ weight
            if ctx.needs_input_grad[1]:
                x = expand(Compressed(*kept, *ctx.how))
                grad_weight = rows.t() @ x.view(-1, x.shape[-1])
            if ctx.needs_input_grad[2]:
                grad_bias = rows.sum(0)
        if not torch.is_grad_enabled():
            return grad_x, grad_weight, grad_bias
        return tuple(_native().first_order([grad_x, grad_weight, grad_bias]))


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``x @ weight.t() + bias`` with ``x`` kept in 8 bits for the gradient of
    ``weight``, which is a matrix product with the expanded copy (that of ``x``
    needs the weight alone). One type for all, that of the result too: autocast does
    not reach the product, with a gradient or without.

    Each call keeps a copy of its own: products of one input (queries, keys and
    values; gate and up) belong in one call with their weights stacked. Three calls
    keep 3.19 bytes an element, where the bfloat16 tensor itself, kept once, has 2."""
    _check_tangent(x, weight, bias)
    if x.dtype != weight.dtype or (bias is not None and bias.dtype != x.dtype):
        raise TypeError(f"x, weight and bias must be of one type, not {x.dtype}, {weight.dtype}" +
                        (f" and {bias.dtype}" if bias is not None else ""))
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias)):
        return _Linear.apply(x, weight, bias)
    with torch.autocast("cuda", enabled=False):
        return torch.nn.functional.linear(x, weight, bias)
