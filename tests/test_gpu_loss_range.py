"""The losses over the whole range of finite logits and temperatures: masks that
are large finite numbers, rows far from zero, temperatures from 2^-20 to 2^20."""
import pytest
import torch

from quantized_optimizer_state_gb300 import fo
from tests.test_gpu_logprobs import check_forward

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


@pytest.mark.parametrize("temperature,first,then", [(83.0, -55840.0, -55584.0), (71.0, -57216.0, -56960.0), (78.0, -56416.0, -56160.0),
                                                    (63.0, -58112.0, -57856.0)])
def test_sums_carried_over_from_the_edge_of_fp16(temperature, first, then):
    """What a thread has summed beside a reference that is treated with care, FP16's lowest value being near, keeps its
    size when the reference moves to a number that needs none: (m - m') c, and not the difference of rounded products."""
    n, v = 310, 20000                         # one CTA of 256 threads a row
    x = torch.full((n, v), first, dtype=F16, device="cuda")
    x[:, 8192:8192 + 2048:8] = then           # one for each thread, after its first 32 elements
    check_forward(x, torch.full((n,), 8192, device="cuda"), 0, temperature)
