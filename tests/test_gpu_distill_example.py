"""The distillation example: teacher's alternatives, loss with gradient and the
fused optimizer together."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [1009, 50257])
def test_student_learns_the_teacher(vocab):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_optimizer_state_gb300 import distill_example
    r = distill_example.run(vocab=vocab, batch=256, steps=60)
    assert all(math.isfinite(v) for v in r.values())
    assert r["kl_last"] < 0.25 * r["kl_first"]
    assert r["logp_after"] > r["logp_before"] + 1.0
