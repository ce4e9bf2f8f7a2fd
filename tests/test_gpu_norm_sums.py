"""Sums of the norm: long rows of numbers of one sign, whose roundings add up, and the weight's gradient over rows.

u = 2^-24. A sum of n positive terms added one by one is off by up to n u, and for like terms by a good part of it:
they are all rounded the same way. Sums of parts that keep what their roundings lost are off by a few u, whatever n."""
import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo
from tests import act_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
u = 2.0 ** -24

# 1 / rms: the squares' sum of long rows 2 u (of a thread) and 8 additions of threads and warps, the mean's product u, halved
# by the root, and the root's own 2 u: below 8 u. A row in registers: up to 16 squares a lane pair one after another, 5
# additions of lanes, 9 of warps, the mean: (16 + 14 + 1) / 2 + 2 below 18 u.
SUM = {True: 8 * u, False: 18 * u}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


def rows(n, w, spread, seed=0):
    """Positive numbers of one size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1.37 * (1 + spread * torch.rand((n, w), generator=g, device="cuda"))).contiguous()


@pytest.mark.parametrize("spread", [0.0, 0.01, 1.0])
@pytest.mark.parametrize("n,w", [(2, 4096), (1, 16384), (3, 16385), (2, 131072), (2, 1 << 20), (1, 20_000_011)])
def test_long_rows_of_one_sign(n, w, spread):
    x = rows(n, w, spread)
    y, kept = A.rms_norm_forward(x, eps=1e-6)
    r = ref.inverse_rms(x, 1e-6)
    err = SUM[w > 16384]
    assert ((kept.inv_rms.double()[:, None] / r - 1).abs() <= err).all()
    want = x.double() * r
    assert ((y.double() - want).abs() <= want * (err + 2 * u)).all()
    # the gradient's mean: dy of one sign, r as the call saw it
    dy = rows(n, w, spread, seed=1)
    grad, _ = A.rms_norm_backward(kept, dy)
    r = kept.inv_rms.double()[:, None]
    h = ref.kept(x) * r
    mean = (dy.double() * h).mean(1, keepdim=True)
    want = r * (dy.double() - h * mean)
    # h's u, the products' and the sum's as above, twice (no root halves it), and the last three roundings
    assert ((grad.double() - want).abs() <= r * (h * mean * (2 * err + 4 * u) + dy.double() * 4 * u)).all()


@pytest.mark.parametrize("n,w", [(300, 16385), (3, 20000), (300, 768), (4000, 128)])
def test_infinities_in_sums(n, w):
    """They go through the sums as infinities, not as NaN."""
    x, dy = rows(n, w, 1.0), rows(n, w, 1.0, seed=1)
    dy[1, 5] = float("inf")
    _, kept = A.rms_norm_forward(x, torch.ones(w, device="cuda"))
    grad, gw = A.rms_norm_backward(kept, dy)
    assert torch.isinf(gw[5]) and torch.isfinite(gw[:5]).all() and torch.isfinite(gw[6:]).all()
    assert torch.isnan(grad[1, 5]) and (grad[1, :5] == -float("inf")).all() and torch.isfinite(grad[0]).all()


@pytest.mark.parametrize("w", [64, 768, 5003, 20000])
def test_normed_codes_are_rounded_once(w):
    """FP32: with one row and dy = 1 the weight's gradient is h = x^ r itself."""
    g = torch.Generator(device="cuda").manual_seed(w)
    x = torch.randn((1, w), generator=g, device="cuda")
    _, kept = A.rms_norm_forward(x, torch.ones(w, device="cuda"))
    _, h = A.rms_norm_backward(kept, torch.ones_like(x))
    assert torch.equal(h, (ref.kept(x) * kept.inv_rms.double()[:, None]).float()[0])


@pytest.mark.parametrize("w", [768, 4096, 20000])
def test_weights_gradient_keeps_small_terms_beside_large_ones(w):
    """dy of +-2^30 in two of 128 rows, each of which a CTA sums by itself, and ones between them: the sum of the ones'
    h is what is left."""
    n = 128
    x = torch.ones(n, w, device="cuda")
    dy = torch.zeros(n, w, device="cuda")
    dy[1:-1:7] = 1.0
    weight = torch.ones(w, device="cuda")
    _, kept = A.rms_norm_forward(x, weight)
    r = kept.inv_rms.double()
    assert (r == r[0]).all()
    few = dy.clone()
    dy[0], dy[n - 1] = 2.0 ** 30, -2.0 ** 30
    _, got = A.rms_norm_backward(kept, dy)
    _, want = A.rms_norm_backward(kept, few)
    exact = (few.double() * (ref.kept(x) * r[:, None]).float().double()).sum(0)
    assert ((want.double() - exact).abs() <= 2 * u * exact).all()
    assert ((got.double() - exact).abs() <= 4 * u * exact).all()
