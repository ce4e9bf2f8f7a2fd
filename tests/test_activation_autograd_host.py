"""Derivatives that the operators on activations do not have, refused before anything reaches a GPU."""
import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo


class Doubled(torch.autograd.Function):
    """2 x, its backward pass through the module's guard."""

    @staticmethod
    def forward(ctx, x):
        return 2 * x

    @staticmethod
    def backward(ctx, g):
        with torch.no_grad():
            grads = [2 * g, None]
        return fo.native().first_order(grads)[0]


def test_gradients_of_a_differentiated_backward_pass_refuse():
    x = torch.ones(3, requires_grad=True)
    g, = torch.autograd.grad(Doubled.apply(x).sum(), x, create_graph=True)
    assert g.requires_grad and torch.equal(g.detach(), torch.full((3,), 2.0))
    with pytest.raises(RuntimeError, match="first derivatives"):
        (g.sum() + (x * x).sum()).backward()
    g, = torch.autograd.grad(Doubled.apply(x).sum(), x)
    assert not g.requires_grad
    x.grad = None
    Doubled.apply(x).sum().backward()
    assert torch.equal(x.grad, torch.full((3,), 2.0)) and not x.grad.requires_grad


def test_tangents_of_incoming_gradients_are_refused():
    x = torch.zeros(4, 64)
    kept = A.KeptActivation("silu", torch.zeros(4 * 68, dtype=torch.int8), torch.Size((4, 64)), torch.float32, False)
    norm = A.KeptNorm(torch.zeros(4 * 72, dtype=torch.int8), torch.Size((4, 64)), torch.float32, None)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, x)
        for call in (lambda: A.activation_backward(kept, dual), lambda: A.rms_norm_backward(norm, dual),
                     lambda: A.rms_norm_backward(norm._replace(weight=dual[0]), x)):
            with pytest.raises(NotImplementedError, match="tangent"):
                call()
