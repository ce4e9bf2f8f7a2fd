"""Losses on the logits of a language model, with their gradients, through the
library's kernels: what stands between a model's head and the optimizers of
:mod:`.optim`.

* :func:`token_logprobs` -- log probabilities of given tokens, entropies and
  top alternatives; differentiable (policy training, cross entropy). Its
  alternatives are what a teacher hands to
* :func:`distill_loss` -- KL divergence from a teacher known by its top
  logits; differentiable;
* :func:`distill_loss_grad` -- the same loss with its gradient in one call: the
  logits are read once and the gradient written once, where loss and backward
  pass read them twice. For training loops that know the weight of each row
  beforehand: ``loss, grad = distill_loss_grad(...); logits.backward(grad)``.

Logits are bfloat16, float16 or float32 CUDA tensors ``[..., vocab]`` whose
last dimension is contiguous; a slice like ``logits[:, :-1]`` is read where it
lies. The rules for masked, infinite and invalid entries stand in
``include/fo.h``. Work is enqueued on the current stream.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from . import fo


class TokenLogprobs(NamedTuple):
    logp: Optional[torch.Tensor]       # [...], None without tokens
    entropy: Optional[torch.Tensor]    # [...], None with entropy=False
    top_ids: Optional[torch.Tensor]    # [..., top_k] int32, descending, None with top_k=0
    top_logp: Optional[torch.Tensor]   # [..., top_k]


def _check_rows(name: str, x: Optional[torch.Tensor], shape) -> None:
    if x is not None and x.shape != shape:
        raise ValueError(f"{name} must have the logits' leading shape {tuple(shape)}, not {tuple(x.shape)}")


def _aligned_like(logits: torch.Tensor) -> torch.Tensor:
    """An uninitialised gradient for ``logits`` whose rows start at the same
    alignment (modulo 16 bytes), so that the kernels' vectors of both line up:
    rows of an odd vocabulary in a padded matrix would otherwise not. At most
    7 elements are added to a row."""
    if logits.dim() == 2 and logits.shape[0] > 1 and logits.stride(0) > logits.shape[1]:
        per_16 = 16 // logits.element_size()
        pitch = logits.shape[1] + (logits.stride(0) - logits.shape[1]) % per_16
        return torch.empty((logits.shape[0], pitch), dtype=logits.dtype,
                           device=logits.device)[:, :logits.shape[1]]
    return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)


def _on_device_of(x: torch.Tensor):
    """Backward passes run on autograd's threads: the library's calls launch on the current device."""
    return contextlib.nullcontext() if x.device.index == torch.cuda.current_device() else torch.cuda.device(x.device)


def _logprobs(logits, tokens, top_k, temperature, entropy, stats):
    rows, dev, f32 = logits.shape[:-1], logits.device, torch.float32
    logp = torch.empty(rows, dtype=f32, device=dev) if tokens is not None else None
    ent = torch.empty(rows, dtype=f32, device=dev) if entropy else None
    top_ids = torch.empty(rows + (top_k,), dtype=torch.int32, device=dev) if top_k else None
    top_logp = torch.empty(rows + (top_k,), dtype=f32, device=dev) if top_k else None
    fo.fo_token_logprobs(logits, tokens, top_k, logp, ent, top_ids, top_logp, stats, temperature)
    return logp, ent, top_ids, top_logp


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top_k, temperature, entropy):
        stats = torch.empty(logits.shape[:-1] + (fo.FO_LOSS_STATS,), dtype=torch.float32, device=logits.device)
        out = _logprobs(logits, tokens, top_k, temperature, entropy, stats)
        ctx.save_for_backward(logits, tokens, out[2], stats)
        ctx.temperature = temperature
        if top_k:
            ctx.mark_non_differentiable(out[2])
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logp, g_entropy, _, g_top):
        logits, tokens, top_ids, stats = ctx.saved_tensors
        grad = _aligned_like(logits)
        with _on_device_of(logits):
            fo.fo_token_logprobs_grad(logits, stats, grad, tokens, _dense(g_logp), _dense(g_entropy), top_ids,
                                      _dense(g_top), 0 if top_ids is None else top_ids.shape[-1], ctx.temperature)
        return grad, None, None, None, None


def _dense(g: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if g is None else g.contiguous()


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, top_k: int = 0,
                   temperature: float = 1.0, entropy: bool = True) -> TokenLogprobs:
    """Log probabilities under ``softmax(logits / temperature)``, in float32.

    ``tokens``: int64 ids, of the logits' leading shape; a negative one (a
    position to ignore) has log probability 0 and no gradient. ``top_k``: the
    number of most probable tokens to list (up to 128), equal logits by
    ascending id. Differentiable in the logits through ``logp``, ``entropy``
    and ``top_logp``.
    """
    if tokens is not None:
        _check_rows("tokens", tokens, logits.shape[:-1])
        tokens = tokens.contiguous()
    if top_k and (not 0 < top_k <= fo.FO_MAX_TOP_K or (top_k > logits.shape[-1] and logits.numel())):
        raise ValueError(f"top_k must be in 0..{min(fo.FO_MAX_TOP_K, logits.shape[-1])}, not {top_k}")
    if logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, top_k, float(temperature), bool(entropy)))
    return TokenLogprobs(*_logprobs(logits, tokens, top_k, float(temperature), entropy, None))


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, lse, temperature, teacher_temperature, tail):
        rows, dev = logits.shape[:-1], logits.device
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
        stats = torch.empty(rows + (fo.FO_LOSS_STATS,), dtype=torch.float32, device=dev)
        fo.fo_distill(logits, ids, teacher, lse, None, loss, stats, None, temperature, teacher_temperature, tail)
        ctx.save_for_backward(logits, ids, teacher, lse, stats)
        ctx.how = (temperature, teacher_temperature, tail)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss):
        logits, ids, teacher, lse, stats = ctx.saved_tensors
        grad = _aligned_like(logits)
        with _on_device_of(logits):
            fo.fo_distill_grad(logits, ids, teacher, stats, g_loss.contiguous(), grad, lse, *ctx.how)
        return grad, None, None, None, None, None, None


def _check_teacher(logits, ids, teacher, lse) -> None:
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
    ids, teacher = teacher_ids.contiguous(), teacher_logits.detach().contiguous()
    lse = None if teacher_lse is None else teacher_lse.detach().contiguous()
    how = (float(temperature), float(teacher_temperature), bool(tail))
    if logits.requires_grad and torch.is_grad_enabled():
        return _Distill.apply(logits, ids, teacher, lse, *how)
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    fo.fo_distill(logits, ids, teacher, lse, None, loss, None, None, *how)
    return loss


def distill_loss_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                      row_weight: Optional[torch.Tensor] = None, temperature: float = 1.0,
                      teacher_temperature: float = 1.0, tail: bool = False,
                      teacher_lse: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """``(loss, grad)``: ``loss = row_weight * distill_loss(...)`` by position and
    the gradient of its sum with respect to the logits, in one pass.

    ``row_weight`` (float32, 1 where None): for a mean over n tokens 1 / n, and
    0 for padding, whose logits are then not read. ``out``: where to write the
    gradient; it may be ``logits`` itself, which the gradient then replaces.
    """
    _check_teacher(logits, teacher_ids, teacher_logits, teacher_lse)
    _check_rows("row_weight", row_weight, logits.shape[:-1])
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    grad = _aligned_like(logits) if out is None else out
    fo.fo_distill(logits, teacher_ids.contiguous(), teacher_logits.contiguous(), _dense(teacher_lse), _dense(row_weight),
                  loss, None, grad, float(temperature), float(teacher_temperature), bool(tail))
    return loss, grad
