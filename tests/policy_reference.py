"""The policy loss in 64 bits, from its definition, with tolerances.

A log probability l is within t = 2^-19 + 4 u (|d| + ln Z) (tests/loss_reference.py;
u = 2^-24). The ratio q = exp(l - old) has that error, the rounding of l and of the
difference, and the exponential's 2 u: q (t + u (|l| + |l - old|) + 2 u); the loss
A q two more roundings. The KL term b (e^k - k - 1), k = ref - l, has
|e^k - 1| (t + u (|l| + |k|)) from k and 4 u of its terms' sizes (of its own size
where |k| < 1/2: a series); its slope b (1 - e^k) the same with e^k for e^k - 1.
A gradient: the slope's error, and 2^-18 of the probabilities.
"""
import math

import torch

from tests import loss_reference as ref

u = 2.0 ** -24


def policy(x, tokens, old, adv, lo=0.2, hi=0.2, ref_logp=None, beta=0.0, temperature=1.0, weight=None):
    """(loss, logp, grad), each with its tolerance, for every row."""
    n, v = x.shape
    d, p, lp, lnz = ref.row_stats(x, temperature)
    there, bad = tokens >= 0, tokens >= v
    at = tokens.clamp(0, v - 1)[:, None]
    l = torch.where(bad, torch.full_like(lnz[:, 0], math.nan), lp.gather(1, at)[:, 0])
    t = 2.0 ** -19 + 4 * u * (d.gather(1, at)[:, 0].abs() + lnz[:, 0].abs())
    t = torch.where(torch.isfinite(t), t, torch.zeros_like(t))
    old, a = old.double(), adv.double()
    q = (l - old).exp()
    q_err = q * (t + u * (l.abs() + (l - old).abs()) + 2 * u)
    q_err = torch.where(q == 0, torch.zeros_like(q), q_err)      # l - old = -inf: q is 0 exactly, not 0 times infinity
    inside = torch.where(a >= 0, q <= 1 + hi, q >= 1 - lo)
    bound = torch.where(inside, q, torch.where(a >= 0, torch.full_like(q, 1 + hi), torch.full_like(q, 1 - lo)))
    zero = torch.zeros_like(q)
    loss = torch.where(a == 0, zero, -bound * a)
    slope = torch.where((a == 0) | ~inside, zero, -a * q)
    loss_err = torch.where(a == 0, zero, a.abs() * (torch.where(inside, q_err, zero) + 2 * u * bound))
    slope_err = torch.where((a == 0) | ~inside, zero, a.abs() * (q_err + 2 * u * q))
    nan = ((a != 0) & (torch.isnan(q) | torch.isnan(a)))
    loss, slope = torch.where(nan, q * math.nan, loss), torch.where(nan, q * math.nan, slope)
    if beta:
        k = ref_logp.double() - l
        e = k.exp()
        kl = torch.where(k == math.inf, k, torch.expm1(k) - k)
        k_err = torch.where(torch.isfinite(k), t + u * (l.abs() + k.abs()), zero)   # e^-inf is 0 exactly
        loss, slope = loss + beta * kl, slope - beta * torch.expm1(k)
        own = torch.where(k.abs() < 0.5, kl, e + k.abs() + 1)
        loss_err = loss_err + beta * (torch.expm1(k).abs() * k_err + k_err ** 2 + 6 * u * own) + u * loss.abs()
        slope_err = slope_err + beta * (e * k_err + 4 * u * torch.expm1(k).abs()) + u * slope.abs()
    w = torch.ones_like(q) if weight is None else weight.double()
    off = ~there | (w == 0)
    l = torch.where(off, zero, l)
    loss, slope = torch.where(off, zero, loss * w), torch.where(off, zero, slope * w)
    loss_err, slope_err = torch.where(off, zero, (loss_err + u * loss.abs()) * w.abs()), torch.where(off, zero, slope_err * w.abs())
    own = torch.zeros_like(p).scatter_(1, at, 1.0)
    empty = (p.sum(1) == 0)[:, None]
    # what is not finite, as a number of FP32, makes the gradient NaN
    slope = torch.where(torch.isfinite(slope.float()), slope, slope * math.nan + math.nan)[:, None]
    grad = torch.where(empty | off[:, None], torch.zeros_like(p), slope * (own - p)) / temperature
    err = (slope_err[:, None] * (own - p).abs() + slope.abs() * (2.0 ** -18 * p + 4 * u * own)) / temperature
    return (loss, loss_err), (l, torch.where(off, zero, t + u * l.abs())), (grad, torch.nan_to_num(err, nan=0.0, posinf=0.0))


def close(got, want, tol, what):
    dt = got.dtype
    tol = torch.nan_to_num(tol, nan=0.0, posinf=0.0)
    ref.close(got, want, tol + ref.UNIT[dt] * want.abs().nan_to_num(posinf=0.0) * (1 + 2.0 ** -6) + ref.TINY[dt], what)
