"""The losses from several host threads at once, each on its own stream and buffers: calls of one kernel with
different needs of shared memory do not disturb one another."""
import ctypes
import threading

import pytest
import torch

from quantized_optimizer_state_gb300 import fo
from tests.test_gpu_distill import make_teacher
from tests.test_gpu_logprobs import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


class Call:
    """A C call whose arguments are made beforehand, so that threads spend their time in the library and not under
    the interpreter's lock; `out` are the tensors that it writes."""

    def __init__(self, name, out, *args):
        self.f, self.out, self.stream = getattr(fo.lib(), name), out, torch.cuda.Stream()
        self.kept = args
        self.args = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args] + [self.stream.cuda_stream]

    def __call__(self):
        return self.f(*self.args)


def distill(x, ids, y, with_grad):
    n, v = x.shape
    loss, grad = torch.zeros(n, device="cuda"), torch.zeros_like(x) if with_grad else None
    t = fo._teacher(ids, y, None, n, 1.0, False, x.device.index)
    return Call("fo_distill", [loss] + ([grad] if with_grad else []), fo.logits_rows(x), t, None, loss.data_ptr(), None,
                fo.FoLogitsGrad(grad.data_ptr(), v, 0) if with_grad else None)


def alternatives(x, k):
    n = x.shape[0]
    ids, top = torch.zeros(n, k, dtype=torch.int32, device="cuda"), torch.zeros(n, k, device="cuda")
    return Call("fo_token_logprobs", [ids, top], fo.logits_rows(x), None, k, None, None, ids.data_ptr(), top.data_ptr(), None)


def side_by_side(calls, times):
    """Each call once alone, then `times` times in a thread of its own: no call fails and the results are the same."""
    want = []
    torch.cuda.synchronize()
    for call in calls:
        assert call() == 0
        call.stream.synchronize()
        want.append([t.clone() for t in call.out])
        for t in call.out:
            t.zero_()
    torch.cuda.synchronize()
    start, status = threading.Barrier(len(calls)), [set() for _ in calls]

    def work(i):
        start.wait()
        for _ in range(times):
            status[i].add(calls[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{0}] * len(calls)
    for call, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(call.out, w))


def test_distillation_with_and_without_gradient():
    """The fused call needs room for its marks beside the stages, the loss alone does not; vocabularies differ too."""
    calls, kept = [], []
    for v in (50257, 128256):
        x = make(2, v, F32, seed=v)
        ids, y, _ = make_teacher(2, v, 8)
        kept.append((x, ids, y))
        calls += [distill(x, ids, y, True), distill(x, ids, y, False)]
    side_by_side(calls, 10000)


def test_alternatives_of_different_vocabularies():
    """A row's group maxima take 32 KB and more of shared memory on long rows of a CTA of their own."""
    xs = [make(310, v, dtype, seed=v) for v, dtype in ((400000, F32), (330000, F32), (200000, F32))]
    side_by_side([alternatives(x, 5) for x in xs], 500)
