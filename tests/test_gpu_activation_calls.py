"""Operators on activations as calls of a program: under autocast, beside other Python threads, twice differentiated, and
what a graph holds of them."""
import gc
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


def test_other_threads_run_while_a_call_waits_for_the_queue():
    """A launch waits where the stream's queue is full: other Python threads go on meanwhile."""
    x = make((4, 64), BF)
    kept = A.compress(x)
    torch.cuda.synchronize()
    stream, calls, done = torch.cuda.Stream(), 6000, []

    def work():
        with torch.cuda.stream(stream):
            torch.cuda._sleep(2_000_000_000)           # about a second
            begin = time.perf_counter()
            for _ in range(calls):
                A.expand(kept, out=x)
            done.append(time.perf_counter() - begin)

    thread = threading.Thread(target=work)
    thread.start()
    gap, last = 0.0, time.perf_counter()
    while thread.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        gap, last = max(gap, now - last), now
    thread.join()
    torch.cuda.synchronize()
    assert done and done[0] > 0.5, "the queue was never full"
    assert gap < 0.5 * done[0], f"this thread stood still for {gap:.2f} of {done[0]:.2f} s"


def held(make_graph, expected, tensors):
    """That what make_graph returns keeps the expected bytes allocated (the allocator rounds a tensor up by less than 1 MB)."""
    gc.collect()                                       # what earlier tests left is not freed in between
    before = torch.cuda.memory_allocated()
    keep = make_graph()
    over = torch.cuda.memory_allocated() - before - expected
    del keep
    assert 0 <= over < tensors << 20, f"{over} bytes more than {expected}"


def test_what_a_graph_holds():
    """Of its input an operator keeps 1.0625 bytes an element (a norm 4 more a row), and each product a copy of its own."""
    n, w = 8192, 4096
    y, kept = n * w * 2, n * w * 34 // 32
    wide = make((n, 2 * w), BF).requires_grad_(True)
    x = wide.detach()[:, :w].contiguous().requires_grad_(True)
    held(lambda: A.activation(x, "gelu"), y + kept, 2)
    held(lambda: A.activation(wide, "swiglu"), y + 2 * kept, 2)
    held(lambda: A.rms_norm(x), y + kept + 4 * n, 2)
    held(lambda: A.activation(x.detach(), "gelu"), y, 1)
    weights = [make((w, w), BF, seed=i, scale=0.01).requires_grad_(True) for i in (1, 2, 3)]
    A.linear(x, weights[0])                            # the matrix library's workspace is there
    held(lambda: A.linear(x, weights[0]), y + kept, 3)
    held(lambda: [A.linear(x, m) for m in weights], 3 * (y + kept), 9)
    with torch.no_grad():
        held(lambda: A.linear(x, weights[0]), y, 1)


def test_saved_tensors_go_through_hooks():
    """What a graph keeps can be moved elsewhere meanwhile, by hooks in Python that the calls wait for."""
    x, w, m = (make(s, BF, seed=i).requires_grad_(True) for i, s in enumerate([(6, 128), (128,), (16, 64)]))
    t, zero = torch.arange(6, device="cuda"), torch.zeros(6, device="cuda")

    def grads():
        y = A.linear(A.activation(A.rms_norm(x, w), "swiglu"), m)
        return torch.autograd.grad(policy_loss(y, t, zero - 3, zero + 1).loss.sum(), (x, w, m))

    want, packed = grads(), []

    def pack(a):
        packed.append(a)
        return a.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda a: a.cuda()):
        got = grads()
    assert len(packed) >= 8 and all(torch.equal(p, q) for p, q in zip(got, want))
