"""The policy loss's host side: argument errors of the C calls and the binding's checks. No call here reaches a GPU."""
import ctypes
import math

import pytest
import torch

from quantized_optimizer_state_gb300 import fo, losses
from tests import policy_reference as ref

NULL, MISALIGNED, SIZE, BAD, ALIAS = 1, 2, 3, 4, 7
MB = 1 << 20


def logits(**over):
    base = dict(data=64 * MB, rows=4, vocab=1000, row_stride=1000, inner_rows=4, outer_stride=0, temperature=1.0, dtype=0, reserved=0)
    base.update(over)
    return fo.FoLogits(**base)


def sampled(**over):
    base = dict(tokens=1 * MB, old_logp=2 * MB, advantages=3 * MB, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_weight=0.0)
    base.update(over)
    return fo.FoPolicy(**base)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def loss(x, p=None, weight=None, loss=4 * MB, logp=5 * MB, stats=None, grad=None):
    return fo.lib().fo_policy_loss(_ref(x), _ref(p), weight, loss, logp, stats, _ref(grad), None)


def loss_grad(x, tokens=1 * MB, stats=6 * MB, g=7 * MB, grad=None):
    return fo.lib().fo_policy_loss_grad(_ref(x), tokens, stats, g, _ref(grad), None)


GRAD = dict(data=128 * MB, row_stride=1000, outer_stride=0)


@pytest.mark.parametrize("call", [lambda x: loss(x, sampled()), lambda x: loss_grad(x, grad=fo.FoLogitsGrad(**GRAD))])
def test_logits_are_checked(call):
    assert call(None) == NULL and call(logits(data=None)) == NULL
    assert call(logits(rows=-1)) == SIZE and call(logits(vocab=0)) == SIZE and call(logits(vocab=fo.FO_MAX_ROW_BYTES)) == SIZE
    assert call(logits(dtype=3)) == BAD and call(logits(temperature=0.0)) == BAD and call(logits(row_stride=-1)) == BAD
    assert call(logits(data=64 * MB + 1)) == MISALIGNED
    assert call(logits(rows=0)) == 0


def test_policy_arguments():
    x = logits()
    assert ctypes.sizeof(fo.FoPolicy) == 56
    assert loss(x, None) == NULL
    for name in ("tokens", "old_logp", "advantages"):
        assert loss(x, sampled(**{name: None})) == NULL
    assert loss(x, sampled(kl_weight=0.1)) == NULL                     # a KL term without a reference
    for bad in (dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_low=math.nan), dict(clip_high=-0.1), dict(clip_high=math.inf),
                dict(clip_high=math.nan), dict(kl_weight=-1.0), dict(kl_weight=math.nan), dict(kl_weight=math.inf)):
        assert loss(x, sampled(**bad)) == BAD
    assert loss(x, sampled(tokens=MB + 4)) == MISALIGNED and loss(x, sampled(old_logp=2 * MB + 2)) == MISALIGNED
    assert loss(x, sampled(ref_logp=8 * MB + 1, kl_weight=0.1)) == MISALIGNED
    assert loss(x, sampled(), stats=6 * MB + 8) == MISALIGNED and loss(x, sampled(), weight=9 * MB + 1) == MISALIGNED
    assert loss(x, sampled(), loss=2 * MB + 12) == ALIAS and loss(x, sampled(), logp=4 * MB) == ALIAS
    assert loss(x, sampled(ref_logp=4 * MB, kl_weight=0.1)) == ALIAS
    assert loss(x, sampled(), loss=64 * MB + 100) == ALIAS and loss(x, sampled(), weight=5 * MB) == ALIAS
    g = lambda **over: fo.FoLogitsGrad(**{**GRAD, **over})
    assert loss(x, sampled(), grad=g(data=None)) == NULL and loss(x, sampled(), grad=g(row_stride=999)) == BAD
    assert loss(x, sampled(), grad=g(data=64 * MB + 2)) == ALIAS and loss(x, sampled(), grad=g(data=1 * MB)) == ALIAS
    assert loss(x, sampled(), loss=None, logp=None) == 0               # nothing asked for
    assert loss_grad(x, grad=None) == NULL and loss_grad(x, tokens=None, grad=g()) == NULL
    assert loss_grad(x, stats=None, grad=g()) == NULL and loss_grad(x, g=None, grad=g()) == NULL
    assert loss_grad(x, stats=6 * MB + 4, grad=g()) == MISALIGNED and loss_grad(x, stats=128 * MB, grad=g()) == ALIAS


def test_python_refusals(monkeypatch):
    monkeypatch.setattr(fo, "_get_device", lambda: 0)
    x, f = torch.zeros(3, 8), torch.zeros(3)
    t = torch.zeros(3, dtype=torch.long)
    for call in (losses.policy_loss, losses.policy_loss_grad):
        with pytest.raises(ValueError, match="CUDA"):
            call(x, t, f, f)
        with pytest.raises(ValueError, match="tokens"):
            call(x, t[:2], f, f)
        with pytest.raises(ValueError, match="old_logp"):
            call(x, t, f[:, None], f)
        with pytest.raises(ValueError, match="advantages"):
            call(x, t, f, f[:1])
        with pytest.raises(ValueError, match="ref_logp"):
            call(x, t, f, f, ref_logp=f[:1], kl_weight=0.1)
        with pytest.raises(ValueError, match="kl_weight"):
            call(x, t, f, f, kl_weight=0.1)
    with pytest.raises(ValueError, match="row_weight"):
        losses.policy_loss_grad(x, t, f, f, row_weight=f[:2])
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, x)
        with pytest.raises(NotImplementedError, match="tangent"):
            losses.policy_loss(dual, t, f, f)


def test_reference_gradient_against_automatic_differentiation():
    torch.manual_seed(0)
    n, v = 12, 9
    x = torch.randn(n, v, dtype=torch.float64, requires_grad=True)
    t, a = torch.randint(0, v, (n,)), torch.randn(n)
    l = torch.log_softmax(x.detach() / 0.7, 1).gather(1, t[:, None])[:, 0]
    old, r = (l + 0.4 * torch.randn(n)).float(), (l + 0.3 * torch.randn(n)).float()
    lp = torch.log_softmax(x / 0.7, 1).gather(1, t[:, None])[:, 0]
    q, k = (lp - old).exp(), r - lp
    want = -torch.minimum(q * a, q.clamp(0.8, 1.3) * a) + 0.2 * (k.exp() - k - 1)
    loss, logp, grad = ref.policy(x.detach(), t, old, a, 0.2, 0.3, r, 0.2, 0.7)
    assert torch.allclose(loss[0], want) and torch.allclose(logp[0], lp)
    assert torch.allclose(grad[0], torch.autograd.grad(want.sum(), x)[0])
