"""The policy loss by every path that its launch takes, against 64 bits: registers, the ring by two warps, the ring by
eight, clusters, clusters that take a second row; each with padded rows, and with the gradient in the logits' place."""
import pytest
import torch

from quantized_optimizer_state_gb300 import fo
from quantized_optimizer_state_gb300.losses import policy_loss, policy_loss_grad
from tests import policy_reference as ref
from tests.test_gpu_policy import make

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")

# rows by SMs where the launch goes by them
CASES = {
    "registers of a warp": (700, 1000, BF),
    "registers of two warps": (900, 4001, F16),
    "two warps, two rows a CTA": (1300, 6000, BF),
    "two warps, many rows a CTA, no alignment": (4001, 5003, F32),
    "two warps, 32 KB": (2500, 16384, F16),
    "eight warps, one row a CTA": (400, 30011, F32),
    "eight warps, rows in turn": (1500, 20011, BF),
    "clusters of few rows": (5, 128256, BF),
    "clusters of one row, by the cache": (500, 128256, BF),
    "clusters of two rows each": (1000, 262144, BF),
    "clusters of two rows each, no alignment": (1003, 131071, F32),
}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def compare(x, t, old, a, r, w, o, beta):
    """Every row against 64 bits, some rows at a time."""
    n, v = x.shape
    block = max(1, 2 ** 25 // v)
    for i in range(0, n, block):
        s = slice(i, min(i + block, n))
        want = ref.policy(x[s], t[s], old[s], a[s], ref_logp=r[s], beta=beta, weight=w[s])
        for name, got, (value, tol) in zip(("loss", "log probability", "gradient"), o, want):
            ref.close(got[s], value, tol, f"{name}, rows from {i}")


@pytest.mark.parametrize("case", list(CASES))
def test_every_path(case):
    n, v, dtype = CASES[case]
    x, t, old, a, r, w = make(n, v, dtype, seed=n)
    how = dict(ref_logp=r, kl_weight=0.1, row_weight=w)
    whole = policy_loss_grad(x, t, old, a, **how)
    compare(x, t, old, a, r, w, whole, 0.1)
    # the loss alone, which has one pass
    alone = policy_loss(x, t, old, a, ref_logp=r, kl_weight=0.1)
    ones = torch.ones_like(w)
    for i in range(0, n, max(1, 2 ** 25 // v)):
        s = slice(i, min(i + max(1, 2 ** 25 // v), n))
        (value, tol), (logp, logp_tol), _ = ref.policy(x[s], t[s], old[s], a[s], ref_logp=r[s], beta=0.1, weight=ones[s])
        ref.close(alone.loss[s], value, tol, "loss alone")
        ref.close(alone.logp[s], logp, logp_tol, "log probability alone")
    # padded rows, whose logits are not read, leave the others as they were; by token and by weight
    off = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.4
    off[0], off[-1] = True, n > 5
    pad_t, pad_w = torch.where(off, -1, t), torch.where(off, 0.0, w)
    y = torch.where(off[:, None], torch.full_like(x, NAN), x)
    for tokens, weight in ((pad_t, w), (t, pad_w)):
        o = policy_loss_grad(y, tokens, old, a, ref_logp=r, kl_weight=0.1, row_weight=weight)
        for got, want in zip(o, whole):
            assert (got[off] == 0).all() and torch.equal(got[~off], want[~off])
    # in the logits' place
    place = x.clone()
    o = policy_loss_grad(place, t, old, a, out=place, **how)
    assert o.grad is place and all(torch.equal(p, q) for p, q in zip(o, whole))
    place = y.clone()
    o = policy_loss_grad(place, pad_t, old, a, out=place, **how)
    assert (place[off] == 0).all() and torch.equal(place[~off], whole.grad[~off])
    assert torch.equal(o.loss[~off], whole.loss[~off])
