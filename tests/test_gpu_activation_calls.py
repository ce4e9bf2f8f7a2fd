"""Operators on activations as calls of a program: under autocast, beside other Python threads, twice differentiated, and
what a graph holds of them."""
import threading
import time

import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo
from quantized_optimizer_state_gb300.losses import policy_loss
from tests.test_gpu_activations import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


@pytest.mark.parametrize("inside", [F32, BF])
def test_linear_under_autocast_is_the_same_with_and_without_a_gradient(inside):
    x, w, b = make((5, 64), inside), make((24, 64), inside, seed=1), make((24,), inside, seed=2)
    with torch.autocast("cuda", dtype=torch.float16):
        plain = A.linear(x, w, b)
        with torch.no_grad():
            quiet = A.linear(x, w.clone().requires_grad_(True), b)
        trained = A.linear(x, w.clone().requires_grad_(True), b)
    assert plain.dtype == quiet.dtype == trained.dtype == inside
    assert torch.equal(plain, trained) and torch.equal(quiet, trained)


def test_second_derivatives_are_refused_beside_other_terms():
    """A penalty on a gradient, added to a loss that has derivatives of its own: an error, not a gradient without the
    penalty's part."""
    x, w = make((4, 64), F32).requires_grad_(True), make((16, 64), F32, seed=1).requires_grad_(True)
    t, zero = torch.zeros(4, dtype=torch.long, device="cuda"), torch.zeros(4, device="cuda")
    for f in (lambda: A.activation(x, "silu"), lambda: A.activation(x, "swiglu"), lambda: A.rms_norm(x), lambda: A.linear(x, w),
              lambda: policy_loss(x, t, zero, zero + 1, clip_high=1e9, clip_low=1.0).loss):
        g, = torch.autograd.grad(f().sum(), x, create_graph=True)
        loss = (g ** 2).sum() + (x ** 2).sum() + (w ** 2).sum()
        with pytest.raises(RuntimeError, match="first derivatives|once_differentiable"):
            loss.backward()
