"""The loss operators' host side: argument errors of the C calls, the binding's
checks, and the tests' 64-bit reference against formulas written out. No call
here reaches a GPU."""
import ctypes
import math
import os
import re
import types

import pytest
import torch

from quantized_optimizer_state_gb300 import fo
from tests import loss_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, MISALIGNED, SIZE, BAD, ALIAS = 1, 2, 3, 4, 7
MB = 1 << 20


def _logits(**over):
    base = dict(data=64 * MB, rows=4, vocab=1000, row_stride=1000, inner_rows=4, outer_stride=0, temperature=1.0, dtype=0,
                reserved=0)
    base.update(over)
    return fo.FoLogits(**base)


def _teacher(**over):
    base = dict(ids=1 * MB, logits=2 * MB, lse=None, temperature=1.0, k=8, dtype=1, tail=0, reserved=0)
    base.update(over)
    return fo.FoTeacher(**base)


def _grad(data=128 * MB, row_stride=1000, outer_stride=0):
    return fo.FoLogitsGrad(data, row_stride, outer_stride)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def logprobs(x=None, tokens=3 * MB, top_k=0, logp=4 * MB, entropy=5 * MB, ids=None, top=None, stats=None):
    return fo.lib().fo_token_logprobs(_ref(x), tokens, top_k, logp, entropy, ids, top, stats, None)


def logprobs_grad(x=None, tokens=3 * MB, top_k=0, ids=None, stats=6 * MB, g=7 * MB, h=8 * MB, gt=None, grad=None):
    return fo.lib().fo_token_logprobs_grad(_ref(x), tokens, top_k, ids, stats, g, h, gt, _ref(grad), None)


def distill(x=None, t=None, weight=None, loss=4 * MB, stats=None, grad=None):
    return fo.lib().fo_distill(_ref(x), _ref(t), weight, loss, stats, _ref(grad), None)


def distill_grad(x=None, t=None, stats=6 * MB, g=7 * MB, grad=None):
    return fo.lib().fo_distill_grad(_ref(x), _ref(t), stats, g, _ref(grad), None)


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(fo.FoLogits) == 64 and fo.FoLogits.temperature.offset == 48
    assert ctypes.sizeof(fo.FoTeacher) == 48 and fo.FoTeacher.k.offset == 32
    hdr = open(os.path.join(ROOT, "include", "fo.h")).read()
    for name in ("FO_MAX_TOP_K", "FO_LOSS_STATS"):
        assert int(re.search(rf"#define {name} (\d+)", hdr).group(1)) == getattr(fo, name)
    assert re.search(r"#define FO_MAX_ROW_BYTES \((\d+) \* 1024\)", hdr).group(1) == str(fo.FO_MAX_ROW_BYTES // 1024)


@pytest.mark.parametrize("call", [logprobs, lambda x: logprobs_grad(x, grad=_grad()), lambda x: distill(x, _teacher()),
                                  lambda x: distill_grad(x, _teacher(), grad=_grad())])
def test_logits_are_checked_by_every_call(call):
    assert call(None) == NULL
    assert call(_logits(data=None)) == NULL
    assert call(_logits(rows=-1)) == SIZE
    assert call(_logits(rows=fo.FO_MAX_LOGIT_ROWS + 4)) == SIZE
    assert call(_logits(vocab=0)) == SIZE
    assert call(_logits(vocab=fo.FO_MAX_ROW_BYTES // 2 + 1)) == SIZE
    assert call(_logits(vocab=fo.FO_MAX_ROW_BYTES // 4 + 1, dtype=1)) == SIZE
    for t in (0.0, -1.0, math.nan, math.inf, 2.0 ** -21, 2.0 ** 21):
        assert call(_logits(temperature=t)) == BAD
    assert call(_logits(dtype=3)) == BAD and call(_logits(reserved=1)) == BAD
    assert call(_logits(row_stride=-1)) == BAD and call(_logits(inner_rows=3)) == BAD and call(_logits(inner_rows=0)) == BAD
    assert call(_logits(outer_stride=-5)) == BAD
    assert call(_logits(data=64 * MB + 1)) == MISALIGNED and call(_logits(data=64 * MB + 2, dtype=1)) == MISALIGNED
    assert call(_logits(rows=0)) == 0


def test_token_logprobs_arguments():
    x = _logits()
    assert logprobs(x, tokens=None) == NULL
    assert logprobs(x, top_k=5) == NULL and logprobs(x, top_k=5, ids=9 * MB) == NULL
    assert logprobs(x, top_k=-1) == SIZE and logprobs(x, top_k=fo.FO_MAX_TOP_K + 1) == SIZE
    assert logprobs(_logits(vocab=4, row_stride=4), top_k=5, ids=9 * MB, top=10 * MB) == SIZE
    assert logprobs(x, tokens=3 * MB + 4) == MISALIGNED and logprobs(x, logp=4 * MB + 2) == MISALIGNED
    assert logprobs(x, stats=6 * MB + 8) == MISALIGNED
    assert logprobs(x, logp=3 * MB) == ALIAS                     # over the tokens
    assert logprobs(x, entropy=4 * MB + 12) == ALIAS             # the last of logp
    assert logprobs(x, entropy=64 * MB + 7998) == MISALIGNED
    assert logprobs(x, entropy=64 * MB + 7996) == ALIAS          # the last two logits
    assert logprobs(x, tokens=None, logp=None, entropy=None) == 0    # nothing asked for


def test_token_logprobs_grad_arguments():
    x, g = _logits(), _grad()
    assert logprobs_grad(x, grad=None) == NULL and logprobs_grad(x, grad=_grad(data=None)) == NULL
    assert logprobs_grad(x, stats=None, grad=g) == NULL and logprobs_grad(x, tokens=None, grad=g) == NULL
    assert logprobs_grad(x, top_k=4, gt=9 * MB, grad=g) == NULL
    assert logprobs_grad(x, grad=_grad(data=128 * MB + 1)) == MISALIGNED
    assert logprobs_grad(x, grad=_grad(row_stride=999)) == BAD                  # rows overlap
    assert logprobs_grad(x, grad=_grad(row_stride=-1000)) == BAD
    two = _logits(inner_rows=2, row_stride=1000, outer_stride=3000)
    assert logprobs_grad(two, grad=_grad(row_stride=1000, outer_stride=1999)) == BAD
    assert logprobs_grad(x, grad=_grad(data=64 * MB + 2000)) == ALIAS           # shifted over the logits
    assert logprobs_grad(x, grad=_grad(data=64 * MB, row_stride=1001)) == ALIAS  # the same place, other strides
    assert logprobs_grad(x, stats=128 * MB, grad=g) == ALIAS


def test_distill_arguments():
    x, t = _logits(), _teacher()
    assert distill(x, None) == NULL and distill(x, _teacher(ids=None)) == NULL and distill(x, _teacher(logits=None)) == NULL
    assert distill(x, _teacher(k=0)) == SIZE and distill(x, _teacher(k=fo.FO_MAX_TOP_K + 1)) == SIZE
    for bad in (dict(dtype=3), dict(tail=2), dict(reserved=1), dict(temperature=0.0), dict(temperature=math.nan)):
        assert distill(x, _teacher(**bad)) == BAD
    assert distill(x, _teacher(ids=MB + 2)) == MISALIGNED and distill(x, _teacher(lse=3 * MB + 1, tail=1)) == MISALIGNED
    assert distill(x, t, weight=5 * MB + 2) == MISALIGNED
    assert distill(x, t, loss=2 * MB) == ALIAS                                  # over the teacher's logits
    assert distill(x, t, grad=_grad(data=64 * MB + 2)) == ALIAS
    assert distill(x, t, grad=_grad(row_stride=10)) == BAD
    assert distill(x, t, loss=None) == 0
    assert distill_grad(x, t, grad=None) == NULL and distill_grad(x, t, stats=None, grad=_grad()) == NULL
    assert distill_grad(x, t, g=None, grad=_grad()) == NULL
    assert distill_grad(x, t, g=7 * MB + 1, grad=_grad()) == MISALIGNED


def test_refused_calls_launch_nothing():
    before = fo.fo_kernel_launch_count()
    assert logprobs(_logits(rows=-1)) and distill(_logits(), _teacher(k=0))
    assert fo.fo_kernel_launch_count() == before


def test_row_strides_of_views():
    def got(t):
        return fo._row_strides(t, "logits")
    full = torch.empty(3, 17, 101)
    assert got(full) == (51, 51, 101, 0)
    assert got(full[0]) == (17, 17, 101, 0) and got(full[0, 0]) == (1, 1, 101, 0)
    assert got(full[:, :-1]) == (48, 16, 101, 17 * 101)
    assert got(full[:, :, :100]) == (51, 51, 101, 0)
    assert got(full.transpose(0, 1)) == (51, 3, 17 * 101, 101)
    assert got(full[:1, :-1]) == (16, 16, 101, 0)
    assert got(torch.empty(2, 3, 4, 5)) == (24, 24, 5, 0)
    assert got(torch.empty(2, 0, 5))[0] == 0
    assert got(torch.empty(5).expand(7, 5)) == (7, 7, 0, 0)
    with pytest.raises(ValueError, match="contiguous"):
        got(torch.empty(5, 7).t())
    with pytest.raises(ValueError, match="strides"):
        got(torch.empty(4, 6, 8, 10)[:3, :5, :7])


class _Fake:
    """Stands in for a CUDA tensor in checks that run before any call."""

    def __init__(self, dtype, shape, dev=0, addr=1 << 20):
        self.dtype, self.shape, self._addr = dtype, torch.Size(shape), addr
        self.device = types.SimpleNamespace(index=dev)
        self.is_cuda = True

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return self._addr


def test_binding_checks_types_devices_and_lengths(monkeypatch):
    monkeypatch.setattr(fo, "_current_device", lambda: 0)
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    x = _Fake(bf, (4, 100))
    assert fo.logits_rows(x).vocab == 100 and fo.logits_rows(_Fake(torch.float16, (4, 100))).dtype == fo.FO_LOGITS_F16
    with pytest.raises(TypeError, match="logits"):
        fo.logits_rows(_Fake(torch.float64, (4, 100)))
    with pytest.raises(ValueError, match="cuda:1"):
        fo.logits_rows(_Fake(bf, (4, 100), dev=1))
    with pytest.raises(ValueError, match="CUDA"):
        fo.fo_token_logprobs(torch.empty(4, 100))
    with pytest.raises(TypeError, match="tokens"):
        fo.fo_token_logprobs(x, _Fake(i32, (4,)), logp=_Fake(f32, (4,)))
    with pytest.raises(ValueError, match="needs 4"):
        fo.fo_token_logprobs(x, _Fake(i64, (3,)), logp=_Fake(f32, (4,)))
    with pytest.raises(TypeError, match="top_ids"):
        fo.fo_token_logprobs(x, top_k=3, top_ids=_Fake(i64, (4, 3)), top_logp=_Fake(f32, (4, 3)))
    with pytest.raises(ValueError, match="needs 16"):
        fo.fo_token_logprobs(x, stats=_Fake(f32, (4, 3)))
    ids, y = _Fake(i32, (4, 8)), _Fake(f32, (4, 8))
    with pytest.raises(ValueError, match="one shape"):
        fo.fo_distill(x, ids, _Fake(f32, (4, 7)), loss=_Fake(f32, (4,)))
    with pytest.raises(ValueError, match="need 32"):
        fo.fo_distill(x, _Fake(i32, (3, 8)), _Fake(f32, (3, 8)), loss=_Fake(f32, (4,)))
    with pytest.raises(TypeError, match="teacher_ids"):
        fo.fo_distill(x, _Fake(i64, (4, 8)), y, loss=_Fake(f32, (4,)))
    with pytest.raises(TypeError, match="teacher_logits"):
        fo.fo_distill(x, ids, _Fake(torch.float64, (4, 8)), loss=_Fake(f32, (4,)))
    with pytest.raises(ValueError, match="tail"):
        fo.fo_distill(x, ids, y, _Fake(f32, (4,)), loss=_Fake(f32, (4,)))
    with pytest.raises(TypeError, match="grad"):
        fo.fo_distill(x, ids, y, grad=_Fake(f32, (4, 100)))
    with pytest.raises(ValueError, match="shape"):
        fo.fo_distill(x, ids, y, grad=_Fake(bf, (4, 99)))


def test_reference_on_a_row_written_out():
    """Probabilities 1/2, 1/4, 1/4: the numbers by hand."""
    x = torch.tensor([[math.log(2.0), 0.0, 0.0]])
    d, p, lp, lnz = ref.row_stats(x, 1.0)
    assert torch.allclose(p, torch.tensor([[0.5, 0.25, 0.25]], dtype=torch.float64), atol=1e-7)
    assert abs(float(ref.entropy(p, lp)) - 1.5 * math.log(2)) < 1e-7
    g, _ = ref.logprobs_grad(x, 1.0, torch.tensor([0]), torch.ones(1))
    assert torch.allclose(g, torch.tensor([[0.5, -0.25, -0.25]], dtype=torch.float64), atol=1e-7)
    # entropy: -p (ln p + H); ln p = -ln 2 + ..., H = 1.5 ln 2
    g, _ = ref.logprobs_grad(x, 1.0, h=torch.ones(1))
    l2 = math.log(2)
    want = [-0.5 * (-l2 + 1.5 * l2), -0.25 * (-2 * l2 + 1.5 * l2), -0.25 * (-2 * l2 + 1.5 * l2)]
    assert torch.allclose(g, torch.tensor([want], dtype=torch.float64), atol=1e-7)
    # a teacher with 3/4 on id 0 and 1/4 beside its list
    loss, grad, _, _ = ref.distill(x, torch.tensor([[0]], dtype=torch.int32), torch.tensor([[math.log(0.75)]]), tail=True)
    assert abs(float(loss) - (0.75 * math.log(1.5) + 0.25 * math.log(0.5))) < 1e-6
    assert torch.allclose(grad, torch.tensor([[-0.25, 0.125, 0.125]], dtype=torch.float64), atol=1e-6)
    loss, grad, _, _ = ref.distill(x, torch.tensor([[2, 1]], dtype=torch.int32), torch.tensor([[5.0, 5.0]]))
    assert abs(float(loss) - math.log(2)) < 1e-6
    assert torch.allclose(grad, torch.tensor([[0.5, -0.25, -0.25]], dtype=torch.float64), atol=1e-6)


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 9, generator=g, dtype=torch.float64)
    ids = torch.tensor([[1, 4, 4], [0, -1, 8]], dtype=torch.int32)
    y = torch.randn(2, 3, generator=g, dtype=torch.float64) - 2
    h = 1e-5
    for how in (dict(temperature=1.7), dict(tail=True), dict(tail=True, lse=torch.tensor([0.5, 0.1]))):
        grad = ref.distill(x, ids, y, **how)[1]
        for j in range(9):
            e = torch.zeros_like(x)
            e[:, j] = h
            num = (ref.distill(x + e, ids, y, **how)[0] - ref.distill(x - e, ids, y, **how)[0]) / (2 * h)
            assert torch.allclose(grad[:, j], num, atol=1e-8)
