"""What stands before and after each output of the losses stays as it was, at every alignment of the arrays."""
import pytest
import torch

from quantized_optimizer_state_gb300 import fo
from tests import loss_reference as ref
from tests.test_gpu_distill import make_teacher
from tests.test_gpu_logprobs import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


class Guarded:
    """An array of n elements between two regions that nothing may write to, `cut` elements off a 16-byte boundary."""

    def __init__(self, n, dtype, cut):
        self.mark = -12288                        # a number of every type
        self.all = torch.full((n + 2 * GUARD + cut,), self.mark, dtype=dtype, device="cuda")
        self.of = self.all[GUARD + cut:GUARD + cut + n]
        self.lo, self.hi = GUARD + cut, GUARD + cut + n

    def check(self, what):
        assert (self.all[:self.lo] == self.mark).all() and (self.all[self.hi:] == self.mark).all(), f"{what}: written outside"
        assert (self.of != self.mark).all(), f"{what}: not written"


@pytest.mark.parametrize("cut", [0, 1, 2, 3])
@pytest.mark.parametrize("n,v,k,dtype", [(5, 777, 9, BF), (3, 128256, 128, BF), (1, 50257, 5, F32), (900, 1000, 20, BF), (800, 30011, 64, F32),
                                         (4, 40, 40, F32)])
def test_logprobs(n, v, k, dtype, cut):
    x = make(n, v, dtype, seed=v)
    x[0, k // 2:] = -float("inf")                                  # fewer left than are listed
    t = torch.zeros(n, dtype=torch.long, device="cuda")
    logp, entropy, top = Guarded(n, F32, cut), Guarded(n, F32, cut), Guarded(n * k, F32, cut)
    ids, stats = Guarded(n * k, torch.int32, cut), Guarded(n * fo.FO_LOSS_STATS, F32, 0)
    fo.fo_token_logprobs(x, t, k, logp.of, entropy.of, ids.of, top.of, stats.of)
    for what, a in (("logp", logp), ("entropy", entropy), ("top_ids", ids), ("top_logp", top), ("stats", stats)):
        a.check(what)
    assert torch.equal(ids.of.view(n, k).long(), ref.top(x, k))


@pytest.mark.parametrize("cut", [0, 1, 2, 3])
@pytest.mark.parametrize("n,v,k,dtype", [(5, 777, 9, BF), (3, 128256, 128, BF), (1, 50257, 5, F32), (1300, 1000, 20, BF), (500, 30011, 64, F32)])
def test_distillation(n, v, k, dtype, cut):
    x = make(n, v, dtype, seed=v)
    ids, y, lse = make_teacher(n, v, k)
    loss, grad, stats = Guarded(n, F32, cut), Guarded(n * v, dtype, cut), Guarded(n * fo.FO_LOSS_STATS, F32, 0)
    fo.fo_distill(x, ids, y, lse, None, loss.of, stats.of, grad.of.view(n, v), tail=True)
    for what, a in (("loss", loss), ("gradient", grad), ("stats", stats)):
        a.check(what)
    again = Guarded(n * v, dtype, cut)
    fo.fo_distill_grad(x, ids, y, stats.of, torch.ones(n, device="cuda"), again.of.view(n, v), lse, tail=True)
    again.check("gradient from statistics")
