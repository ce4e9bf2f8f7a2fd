"""The loss operators in 64 bits, from their definitions, and the tolerances of
the tests that compare the kernels with them.

Tolerances (u = 2^-24, the FP32 rounding unit; U the rounding unit of the
logits' type). An exponential 2^t, t = (x - m) log2(e) / T, has three roundings
of t, each at most u |t|, and the hardware's 2^-22. Row sums are partial sums of
at most 2^10 terms that are then joined: the roundings of positive terms add up
to 2^10 u in the worst case and to 2^5 u = 2^-19 as a random walk; 2^-19 is
taken. So, with d = (x - m) / T:
  logp     2^-19 + 4 u (|d| + ln Z)
  entropy  2^-18 + 2^-19 (ln Z + |E d|): Z and the weighted sum W each
  a gradient's p_j: relative 2^-18; its value is rounded once to the logits' type.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}
NAN = float("nan")


def row_stats(x: torch.Tensor, temperature: float):
    """d = (x - m) / T, p, ln p, ln Z, for every row, in 64 bits. Rows that are
    all -inf: p = 0, ln p = -inf, ln Z = -inf."""
    s = x.double() / temperature
    m = s.amax(1, keepdim=True)
    d = s - torch.where(m == -math.inf, torch.zeros_like(m), m)
    z = d.exp().sum(1, keepdim=True)
    lnz = z.log()
    lp = torch.where(z == 0, torch.full_like(d, -math.inf), d - lnz)
    return d, lp.exp(), lp, lnz


def plogp(p, lp):
    """p ln p with 0 ln 0 = 0 and NaN kept."""
    return torch.where(p == 0, torch.zeros_like(p), p * lp)


def entropy(p, lp):
    return -plogp(p, lp).sum(1)


def top(x: torch.Tensor, k: int):
    """Ids of the k largest by row: descending, ties by ascending id, NaN largest."""
    y = x.double()
    return torch.sort(y, dim=1, descending=True, stable=True).indices[:, :k]


def logprobs_grad(x, temperature, tokens=None, g=None, h=None, top_ids=None, g_top=None):
    """The gradient and, elementwise, the scale of its p terms (for the tolerance)."""
    d, p, lp, _ = row_stats(x, temperature)
    n, v = x.shape
    zero = torch.zeros(n, dtype=torch.float64, device=x.device)
    sparse = torch.zeros_like(p)
    size = torch.zeros_like(p)           # sizes of the sparse terms
    total, mass = zero.clone(), zero.clone()
    bad = torch.zeros(n, dtype=torch.bool, device=x.device)
    active = torch.zeros(n, dtype=torch.bool, device=x.device)

    def add(ids, w):
        nonlocal total, mass
        for i in range(ids.shape[1]):
            use = (ids[:, i] >= 0) & (w[:, i] != 0)
            bad.logical_or_(use & (ids[:, i] >= v))
            active.logical_or_(use)
            wi = torch.where(use, w[:, i].double(), zero)
            at = ids[:, i].long().clamp(0, v - 1)[:, None]
            sparse.scatter_add_(1, at, wi[:, None])
            size.scatter_add_(1, at, wi[:, None].abs())
            total = total + wi
            mass = mass + wi.abs()

    if g is not None:
        add(tokens[:, None], g[:, None])
    if g_top is not None:
        add(top_ids, g_top)
    hh = zero if h is None else h.double()
    active.logical_or_(hh != 0)
    ent = entropy(p, lp)
    grad = sparse - p * total[:, None]
    scale = p * mass[:, None] + size
    use_h = (hh != 0)[:, None]
    ph = plogp(p, lp) + p * ent[:, None]
    grad = torch.where(use_h, grad - hh[:, None] * ph, grad)
    scale = torch.where(use_h, scale + hh.abs()[:, None] * (plogp(p, lp).abs() + p * ent[:, None].abs() + p), scale)
    grad = torch.where(bad[:, None], torch.full_like(grad, NAN), grad)
    dead = ~active | (p.sum(1) == 0)
    grad = torch.where(dead[:, None], torch.zeros_like(grad), grad)
    return grad / temperature, scale / temperature


def teacher(ids, logits, temperature, tail=False, lse=None):
    """q, ln q, the mass that is not listed; entries with a negative id are none."""
    y = logits.double() / temperature
    y = torch.where(ids >= 0, y, torch.full_like(y, -math.inf))
    if tail:
        norm = torch.zeros(ids.shape[0], 1, dtype=torch.float64, device=ids.device) if lse is None else lse.double()[:, None]
    else:
        norm = torch.logsumexp(y, 1, keepdim=True)
        norm = torch.where(norm == -math.inf, torch.zeros_like(norm), norm)
    lq = y - norm
    q = lq.exp()
    rest = (1 - q.sum(1)).clamp(min=0) if tail else torch.zeros(ids.shape[0], dtype=torch.float64, device=ids.device)
    return q, lq, rest


def distill(x, ids, logits, temperature=1.0, teacher_temperature=1.0, tail=False, lse=None, weight=None):
    """loss, gradient, the loss's tolerance and the scale of the gradient's terms."""
    n, v = x.shape
    d, p, lp, lnz = row_stats(x, temperature)
    q, lq, rest = teacher(ids, logits, teacher_temperature, tail, lse)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    bad = ((ids >= v).any(1)) | torch.isnan(lnz[:, 0])
    at = ids.long().clamp(0, v - 1)
    there = (ids >= 0) & (ids < v)
    zero = torch.zeros_like(q)
    qq = torch.where(there, q, zero)
    term = torch.where(qq > 0, qq * (lq - lp.gather(1, at)), zero)
    loss = term.sum(1)
    size = torch.where(qq > 0, qq * (lq.abs() + lp.gather(1, at).abs() + lnz.abs() + 1), zero).sum(1)
    target = torch.zeros_like(p).scatter_add_(1, at, qq)
    listed = torch.zeros_like(p).scatter_add_(1, at, there.double()) > 0
    total = torch.where((q > 0).any(1), torch.ones_like(rest), torch.zeros_like(rest))
    if tail:
        total = q.sum(1) + rest
        out = torch.where(listed, torch.zeros_like(p), p)
        p_rest = out.sum(1)
        has = rest > 0
        loss = loss + torch.where(has, rest * (rest.log() - p_rest.log()), torch.zeros_like(rest))
        size = size + torch.where(has, rest * (rest.log().abs() + p_rest.log().abs() + lnz[:, 0].abs() + 1), torch.zeros_like(rest)) + 1
        share = torch.where((p_rest > 0) & has, rest / p_rest, torch.zeros_like(rest))[:, None]
        grad = p * total[:, None] - target - out * share
        scale = p * total[:, None] + target + out * share
        # the rest is 1 - sum q: 128 roundings of q, which moves the share of an unlisted token
        scale = scale + out * torch.where(p_rest > 0, 1 / p_rest, torch.zeros_like(rest))[:, None]
    else:
        grad = p * total[:, None] - target
        scale = p * total[:, None] + target
    nan = torch.full_like(loss, NAN)
    loss = torch.where(bad, nan, loss)
    grad = torch.where(bad[:, None], nan[:, None], grad)
    empty = (p.sum(1) == 0)
    grad = torch.where(empty[:, None], torch.zeros_like(grad), grad)
    off = w == 0
    loss = torch.where(off, torch.zeros_like(loss), loss * w)
    grad = torch.where(off[:, None], torch.zeros_like(grad), grad * (w / temperature)[:, None])
    scale = torch.where(off[:, None], torch.zeros_like(scale), scale * (w.abs() / temperature)[:, None])
    return loss, grad, torch.where(off, torch.zeros_like(size), 2.0 ** -18 * (1 + size) * w.abs()), scale


def close(got, want, tol, what):
    """Equal where `want`, as a value of the result's type, is not finite; within tol elsewhere."""
    beyond = want.to(got.dtype).isinf()
    got, want = got.double(), torch.where(beyond, want.to(got.dtype).double(), want.double())
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand_as(want)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    assert torch.isfinite(got[fine]).all(), f"{what}: not finite where it should be"
    off = (got - want).abs()[fine] - tol[fine]
    if off.numel():
        i = int(off.argmax())
        assert float(off[i]) <= 0, (f"{what}: off by {float((got - want).abs()[fine][i]):.3g}, allowed "
                                    f"{float(tol[fine][i]):.3g}, at value {float(want[fine][i]):.6g}")


def grad_tolerance(grad, scale, dtype):
    """One rounding to the type, relative 2^-18 of the terms, the smallest step of the type."""
    g = torch.where(torch.isfinite(grad), grad.abs(), torch.zeros_like(grad))
    s = torch.where(torch.isfinite(scale), scale, torch.zeros_like(scale))
    return UNIT[dtype] * g * (1 + 2.0 ** -6) + 2.0 ** -18 * s * (1 + UNIT[dtype]) + TINY[dtype]
