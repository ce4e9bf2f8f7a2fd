"""Losses on the logits of a language model, with their gradients, through the
library's kernels: what stands between a model's head and the optimizers of
:mod:`.optim`.

* :func:`token_logprobs` -- log probabilities of given tokens, entropies and
  top alternatives; differentiable (policy training, cross entropy). Its
  alternatives are what a teacher hands to
* :func:`distill_loss` -- KL divergence from a teacher known by its top
  logits; differentiable;
* :func:`distill_loss_grad` -- the same loss with its gradient in one call: the
  logits come from device memory once and the gradient goes there once, where
  loss and backward pass fetch them twice. For training loops that know the
  weight of each row beforehand:
  ``loss, grad = distill_loss_grad(...); logits.backward(grad)``;
* :func:`policy_loss`, :func:`policy_loss_grad` -- the clipped loss of policy
  training on sampled tokens, with a KL term, in the same two forms.

Logits are bfloat16, float16 or float32 CUDA tensors ``[..., vocab]`` whose
last dimension is contiguous; a slice like ``logits[:, :-1]`` is read where it
lies. The rules for masked, infinite and invalid entries stand in
``include/fo.h``. Work is enqueued on the current stream. Derivatives are of the
first order and in reverse mode; a tangent of forward mode is refused.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import fo


class TokenLogprobs(NamedTuple):
    logp: Optional[torch.Tensor]       # [...], None without tokens
    entropy: Optional[torch.Tensor]    # [...], None with entropy=False
    top_ids: Optional[torch.Tensor]    # [..., top_k] int32, descending, None with top_k=0
    top_logp: Optional[torch.Tensor]   # [..., top_k]


def _check_rows(name: str, x: Optional[torch.Tensor], shape) -> None:
    if x is not None and x.shape != shape:
        raise ValueError(f"{name} must have the logits' leading shape {tuple(shape)}, not {tuple(x.shape)}")


def _check_tangent(logits: torch.Tensor) -> None:
    """A tensor with a tangent need not require a gradient, and its address carries none."""
    if forward_ad.unpack_dual(logits).tangent is not None:
        raise NotImplementedError("the losses have no forward-mode derivative: logits carry a tangent")


# The functions below hand the C calls the addresses of tensors that they have
# just made themselves; what the caller passes is checked by fo's helpers.

def _empty_grad(logits: torch.Tensor, x: fo.FoLogits):
    """An uninitialised gradient for ``logits`` and its layout. Its rows start at
    the same alignment (modulo 16 bytes) as the logits', so that the kernels'
    vectors of both line up, where these are contiguous from an aligned base or
    the rows of a padded matrix with one (at most 7 elements are added to a row).
    In other layouts of an odd vocabulary the two do not line up, and most rows
    are stored element by element (3.5 times as long)."""
    vocab = x.vocab
    if x.inner_rows == x.rows and x.rows > 1 and x.row_stride > vocab and logits.dim() == 2:
        pitch = vocab + (x.row_stride - vocab) % (16 // logits.element_size())
        grad = torch.empty((x.rows, pitch), dtype=logits.dtype, device=logits.device)[:, :vocab]
        return grad, fo.FoLogitsGrad(grad.data_ptr(), pitch, 0)
    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    return grad, fo.FoLogitsGrad(grad.data_ptr(), vocab, x.inner_rows * vocab)


def _on_device_of(x: torch.Tensor):
    """Backward passes run on autograd's threads: the library's calls launch on the current device."""
    return contextlib.nullcontext() if x.device.index == fo._current_device() else torch.cuda.device(x.device)


def _dense(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if g is None else g.contiguous()


def _logprobs(logits, tokens, top_k, temperature, entropy, rows, with_stats):
    x = fo.logits_rows(logits, temperature)
    dev, f32, empty = logits.device, torch.float32, torch.empty
    logp = ent = top_ids = top_logp = stats = None
    p_tokens = p_logp = p_ent = p_ids = p_top = p_stats = None
    if tokens is not None:
        p_tokens = fo._array(tokens, "tokens", torch.int64, x.rows, dev.index)
        logp = empty(rows, dtype=f32, device=dev)
        p_logp = logp.data_ptr()
    if entropy:
        ent = empty(rows, dtype=f32, device=dev)
        p_ent = ent.data_ptr()
    if top_k:
        top_ids = empty(rows + (top_k,), dtype=torch.int32, device=dev)
        top_logp = empty(rows + (top_k,), dtype=f32, device=dev)
        p_ids, p_top = top_ids.data_ptr(), top_logp.data_ptr()
    if with_stats:
        stats = empty((x.rows, fo.FO_LOSS_STATS), dtype=f32, device=dev)
        p_stats = stats.data_ptr()
    status = fo.lib().fo_token_logprobs(ctypes.byref(x), p_tokens, top_k, p_logp, p_ent, p_ids, p_top, p_stats,
                                        fo._stream(None))
    if status:
        fo._check("fo_token_logprobs", status)
    return logp, ent, top_ids, top_logp, stats


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top_k, temperature, entropy, rows):
        logp, ent, top_ids, top_logp, stats = _logprobs(logits, tokens, top_k, temperature, entropy, rows, True)
        ctx.save_for_backward(logits, tokens, top_ids, stats)
        ctx.temperature = temperature
        if top_k:
            ctx.mark_non_differentiable(top_ids)
        ctx.set_materialize_grads(False)
        return logp, ent, top_ids, top_logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logp, g_entropy, _, g_top):
        logits, tokens, top_ids, stats = ctx.saved_tensors
        with _on_device_of(logits):
            x = fo.logits_rows(logits, ctx.temperature)
            grad, to = _empty_grad(logits, x)
            n, cur, f32 = x.rows, logits.device.index, torch.float32
            k = 0 if top_ids is None else top_ids.shape[-1]
            g_logp, g_entropy, g_top = _dense(g_logp), _dense(g_entropy), _dense(g_top)
            status = fo.lib().fo_token_logprobs_grad(
                ctypes.byref(x), None if tokens is None else tokens.data_ptr(), k,
                None if top_ids is None else top_ids.data_ptr(), stats.data_ptr(), fo._array(g_logp, "g_logp", f32, n, cur),
                fo._array(g_entropy, "g_entropy", f32, n, cur), fo._array(g_top, "g_top", f32, n * k, cur),
                ctypes.byref(to), fo._stream(None))
            if status:
                fo._check("fo_token_logprobs_grad", status)
        return grad, None, None, None, None, None


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, top_k: int = 0,
                   temperature: float = 1.0, entropy: bool = True) -> TokenLogprobs:
    """Log probabilities under ``softmax(logits / temperature)``, in float32.

    ``tokens``: int64 ids, of the logits' leading shape; a negative one (a
    position to ignore) has log probability 0 and no gradient. ``top_k``: the
    number of most probable tokens to list (up to 128), equal logits by
    ascending id. Differentiable in the logits through ``logp``, ``entropy``
    and ``top_logp``.
    """
    _check_tangent(logits)
    rows = logits.shape[:-1]
    if tokens is not None:
        _check_rows("tokens", tokens, rows)
        tokens = tokens.contiguous()
    if top_k and (not 0 < top_k <= fo.FO_MAX_TOP_K or (top_k > logits.shape[-1] and logits.numel())):
        raise ValueError(f"top_k must be in 0..{min(fo.FO_MAX_TOP_K, logits.shape[-1])}, not {top_k}")
    if logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, top_k, temperature, entropy, rows))
    return TokenLogprobs(*_logprobs(logits, tokens, top_k, temperature, entropy, rows, False)[:4])


def _distill(logits, ids, teacher, lse, weight, temperature, teacher_temperature, tail, with_stats, with_grad, out=None):
    x = fo.logits_rows(logits, temperature)
    dev, n = logits.device, x.rows
    t = fo._teacher(ids, teacher, lse, n, teacher_temperature, tail, dev.index)
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=dev)
    grad = to = stats = p_stats = None
    if out is not None:
        grad, to = out, fo._logits_grad(x, logits, out)
    elif with_grad:
        grad, to = _empty_grad(logits, x)
    if with_stats:
        stats = torch.empty((n, fo.FO_LOSS_STATS), dtype=torch.float32, device=dev)
        p_stats = stats.data_ptr()
    status = fo.lib().fo_distill(ctypes.byref(x), ctypes.byref(t),
                                 fo._array(weight, "row_weight", torch.float32, n, dev.index), loss.data_ptr(), p_stats,
                                 None if to is None else ctypes.byref(to), fo._stream(None))
    if status:
        fo._check("fo_distill", status)
    if out is not None:
        fo._modified(out)
    return loss, grad, stats


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, lse, temperature, teacher_temperature, tail):
        loss, _, stats = _distill(logits, ids, teacher, lse, None, temperature, teacher_temperature, tail, True, False)
        ctx.save_for_backward(logits, ids, teacher, lse, stats)
        ctx.how = (temperature, teacher_temperature, tail)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss):
        logits, ids, teacher, lse, stats = ctx.saved_tensors
        temperature, teacher_temperature, tail = ctx.how
        with _on_device_of(logits):
            x = fo.logits_rows(logits, temperature)
            cur = logits.device.index
            t = fo._teacher(ids, teacher, lse, x.rows, teacher_temperature, tail, cur)
            grad, to = _empty_grad(logits, x)
            g_loss = g_loss.contiguous()
            status = fo.lib().fo_distill_grad(ctypes.byref(x), ctypes.byref(t), stats.data_ptr(),
                                              fo._array(g_loss, "g_loss", torch.float32, x.rows, cur), ctypes.byref(to),
                                              fo._stream(None))
            if status:
                fo._check("fo_distill_grad", status)
        return grad, None, None, None, None, None, None


def _check_teacher(logits, ids, teacher, lse) -> None:
    _check_tangent(logits)
    if ids.shape[:-1] != logits.shape[:-1] or teacher.shape != ids.shape:
        raise ValueError(f"teacher_ids and teacher_logits must be [..., k] over the logits' leading shape "
                         f"{tuple(logits.shape[:-1])}, not {tuple(ids.shape)} and {tuple(teacher.shape)}")
    if not 1 <= ids.shape[-1] <= fo.FO_MAX_TOP_K:
        raise ValueError(f"a teacher lists 1..{fo.FO_MAX_TOP_K} ids, not {ids.shape[-1]}")
    _check_rows("teacher_lse", lse, logits.shape[:-1])


def distill_loss(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                 temperature: float = 1.0, teacher_temperature: float = 1.0, tail: bool = False,
                 teacher_lse: Optional[torch.Tensor] = None) -> torch.Tensor:
    """KL(teacher || student) by position, in float32; the student is
    ``softmax(logits / temperature)``.

    ``teacher_ids`` (int32) and ``teacher_logits`` (bfloat16, float16 or
    float32), ``[..., k]``: a teacher's top ids, -1 for an entry that is none,
    and their logits, or log probabilities. The teacher is the softmax of
    ``teacher_logits / teacher_temperature`` over these ids. With ``tail`` it is
    ``exp(teacher_logits / teacher_temperature - teacher_lse)`` (``teacher_lse``
    0 where None: log probabilities), and the rest of both distributions is
    one more outcome. Differentiable in ``logits``; no factor T^2 is applied.
    """
    _check_teacher(logits, teacher_ids, teacher_logits, teacher_lse)
    ids, teacher, lse = teacher_ids.contiguous(), teacher_logits.detach().contiguous(), _dense(teacher_lse)
    if logits.requires_grad and torch.is_grad_enabled():
        return _Distill.apply(logits, ids, teacher, lse, temperature, teacher_temperature, tail)
    return _distill(logits, ids, teacher, lse, None, temperature, teacher_temperature, tail, False, False)[0]


def distill_loss_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                      row_weight: Optional[torch.Tensor] = None, temperature: float = 1.0,
                      teacher_temperature: float = 1.0, tail: bool = False,
                      teacher_lse: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """``(loss, grad)``: ``loss = row_weight * distill_loss(...)`` by position and
    the gradient of its sum with respect to the logits, in one call.

    ``row_weight`` (float32, 1 where None): for a mean over n tokens 1 / n, and
    0 for padding, whatever its logits hold. ``out``: where to write the
    gradient; it may be ``logits`` itself, which the gradient then replaces (and
    a graph that keeps the logits for its own backward pass refuses to run it).
    """
    _check_teacher(logits, teacher_ids, teacher_logits, teacher_lse)
    _check_rows("row_weight", row_weight, logits.shape[:-1])
    return _distill(logits, teacher_ids.contiguous(), teacher_logits.contiguous(), _dense(teacher_lse), _dense(row_weight),
                    temperature, teacher_temperature, tail, False, True, out)[:2]


class PolicyLoss(NamedTuple):
    loss: torch.Tensor       # [...]
    logp: torch.Tensor       # [...], of the tokens; not differentiable


class PolicyLossGrad(NamedTuple):
    loss: torch.Tensor       # [...], times row_weight
    logp: torch.Tensor
    grad: torch.Tensor       # of the logits


def policy_loss(logits: torch.Tensor, tokens: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                clip_low: float = 0.2, clip_high: float = 0.2, ref_logp: Optional[torch.Tensor] = None,
                kl_weight: float = 0.0, temperature: float = 1.0) -> PolicyLoss:
    """The clipped policy loss by position, in float32, and the log probabilities
    ``l`` of ``tokens`` under ``softmax(logits / temperature)``:
    ``-min(q A, clip(q, 1 - clip_low, 1 + clip_high) A)`` with ``q = exp(l - old_logp)``
    and ``A`` the advantage, plus ``kl_weight * (exp(k) - k - 1)`` with
    ``k = ref_logp - l``.

    ``tokens``: int64 ids of the logits' leading shape, negative where there is no
    position (loss, log probability and gradient 0). ``old_logp``, ``advantages``
    and ``ref_logp``: float32 of that shape, constants of the gradient. The loss is
    differentiable in ``logits``.
    """
    _check_tangent(logits)
    if kl_weight and ref_logp is None:
        raise ValueError("kl_weight needs ref_logp")
    return PolicyLoss(*fo.native().policy_loss(logits, tokens, old_logp, advantages, ref_logp, clip_low, clip_high, kl_weight, temperature))


def policy_loss_grad(logits: torch.Tensor, tokens: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                     clip_low: float = 0.2, clip_high: float = 0.2, ref_logp: Optional[torch.Tensor] = None,
                     kl_weight: float = 0.0, temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> PolicyLossGrad:
    """``(loss, logp, grad)``: ``loss = row_weight * policy_loss(...).loss`` by
    position and the gradient of its sum with respect to the logits, in one call:
    ``o = policy_loss_grad(...); logits.backward(o.grad)``.

    ``row_weight`` (float32, 1 where None): for a mean over n tokens 1 / n, and 0
    for padding, whose logits are not read. ``out``: where to write the gradient;
    it may be ``logits`` itself, which the gradient then replaces.
    """
    _check_tangent(logits)
    if kl_weight and ref_logp is None:
        raise ValueError("kl_weight needs ref_logp")
    return PolicyLossGrad(*fo.native().policy_loss_grad(logits, tokens, old_logp, advantages, ref_logp, clip_low, clip_high, kl_weight,
                                                        temperature, row_weight, out))
