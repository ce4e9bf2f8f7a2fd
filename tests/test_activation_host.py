"""The host side of the operators on activations: argument errors of the C calls, the bindings' checks, and the
tests' 64-bit reference against formulas written out. No call here reaches a GPU."""
import ctypes
import math
import os
import re
import types

import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo
from tests import act_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, MISALIGNED, SIZE, BAD, ALIAS = 1, 2, 3, 4, 7
MB = 1 << 20


def rows(data=64 * MB, **over):
    base = dict(data=data, rows=4, width=100, row_stride=100, dtype=0, reserved=0)
    base.update(over)
    return fo.FoRows(**base)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def compress(x, codes=1 * MB, steps=2 * MB):
    return fo.lib().fo_compress(_ref(x), codes, steps, None)


def expand(x, codes=1 * MB, steps=2 * MB):
    return fo.lib().fo_expand(codes, steps, _ref(x), None)


def act(x, up=None, y=None, kind=0, codes=1 * MB, steps=2 * MB, up_codes=None, up_steps=None):
    y = rows(128 * MB) if y is None else y
    return fo.lib().fo_activation(kind, _ref(x), _ref(up), _ref(y), codes, steps, up_codes, up_steps, None)


def act_grad(dy, dx=None, dup=None, kind=0, codes=1 * MB, steps=2 * MB, up_codes=3 * MB, up_steps=4 * MB):
    return fo.lib().fo_activation_grad(kind, codes, steps, up_codes, up_steps, _ref(dy), _ref(dx), _ref(dup), None)


def norm(x, y=None, weight=5 * MB, wtype=0, eps=1e-6, inv=6 * MB, codes=1 * MB, steps=2 * MB):
    y = rows(128 * MB) if y is None else y
    return fo.lib().fo_rms_norm(_ref(x), weight, wtype, eps, _ref(y), inv, codes, steps, None)


def norm_grad(dy, dx=None, weight=5 * MB, wtype=0, inv=6 * MB, gw=7 * MB, ws=8 * MB, codes=1 * MB, steps=2 * MB):
    return fo.lib().fo_rms_norm_grad(codes, steps, inv, weight, wtype, _ref(dy), _ref(dx), gw, ws, None)


def test_layout_matches_the_header():
    hdr = open(os.path.join(ROOT, "include", "fo.h")).read()
    assert re.search(r"#define FO_MAX_ACT_WIDTH \(1 << (\d+)\)", hdr).group(1) == "30" and fo.FO_MAX_ACT_WIDTH == 1 << 30
    assert re.search(r"#define FO_MAX_ACT_GROUPS \(1 << (\d+)\)", hdr).group(1) == "29" and fo.FO_MAX_ACT_GROUPS == 1 << 29
    assert ctypes.sizeof(fo.FoRows) == 40 and fo.FoRows.dtype.offset == 32
    assert re.search(r"FO_ACT_SILU = 0", hdr) and re.search(r"FO_ACT_GELU = 1", hdr)


@pytest.mark.parametrize("call", [compress, expand, act, norm, lambda x: act(rows(), y=x) if x else act(rows(), y=rows(data=None)),
                                  lambda x: act_grad(x, rows(128 * MB)), lambda x: norm_grad(x, rows(128 * MB))])
def test_matrices_are_checked_by_every_call(call):
    assert call(None) == NULL and call(rows(data=None)) == NULL
    assert call(rows(rows=-1)) == SIZE and call(rows(width=0)) == SIZE
    assert call(rows(width=1 << 40)) == SIZE and call(rows(rows=1 << 30, width=1)) == SIZE
    assert call(rows(rows=(1 << 29) // 4 + 1, width=100)) == SIZE
    assert call(rows(dtype=3)) == BAD and call(rows(reserved=1)) == BAD
    assert call(rows(row_stride=-1)) == BAD and call(rows(row_stride=1 << 50)) == BAD
    assert call(rows(data=64 * MB + 1)) in (MISALIGNED, BAD)
    assert call(rows(rows=1 << 27, width=100, row_stride=1 << 40)) in (SIZE, BAD)   # offsets beyond 63 bits; unlike y


def test_empty_matrices_are_no_ops():
    none = rows(data=None, rows=0)
    assert compress(none, None, None) == 0 and expand(none, None, None) == 0
    assert act(none, y=rows(data=None, rows=0)) == 0 and act_grad(none, rows(data=None, rows=0)) == 0
    assert norm(none, rows(data=None, rows=0)) == 0 and norm_grad(none, rows(data=None, rows=0), gw=None) == 0


def test_codes_arguments():
    assert compress(rows(), None) == NULL and compress(rows(), steps=None) == NULL
    assert compress(rows(), MB + 8) == MISALIGNED and compress(rows(), steps=2 * MB + 1) == MISALIGNED
    assert compress(rows(), codes=64 * MB + 784) == ALIAS           # the last 16 of its 800 bytes
    assert compress(rows(), steps=64 * MB - 30) == ALIAS            # 32 bytes of steps
    assert compress(rows(), codes=MB, steps=MB + 510) == ALIAS      # 512 bytes of codes
    assert expand(rows(), codes=64 * MB) == ALIAS
    assert expand(rows(row_stride=99)) == BAD                       # rows that are written overlap
    assert expand(rows(data=64 * MB + 1)) == MISALIGNED and expand(rows(data=64 * MB + 2, dtype=1)) == MISALIGNED


def test_activation_arguments():
    x, y = rows(), rows(128 * MB)
    assert act(x, kind=2) == BAD and act(x, kind=-1) == BAD
    assert act(x, y=rows(128 * MB, rows=5)) == BAD and act(x, y=rows(128 * MB, dtype=2)) == BAD
    assert act(x, up=rows(65 * MB, width=99)) == BAD
    assert act(x, y=rows(128 * MB, row_stride=50)) == BAD
    assert act(x, steps=None) == NULL and act(x, up=rows(65 * MB)) == NULL
    assert act(x, up=rows(65 * MB), up_codes=3 * MB, up_steps=None) == NULL
    assert act(x, y=x) == ALIAS and act(x, up=rows(128 * MB), up_codes=3 * MB, up_steps=4 * MB) == ALIAS
    assert act(x, codes=128 * MB) == ALIAS
    dy, dx = rows(), rows(128 * MB)
    assert act_grad(dy, dx, kind=5) == BAD and act_grad(dy, None) == NULL
    assert act_grad(dy, dx, codes=None) == NULL and act_grad(dy, dx, rows(160 * MB), up_codes=None) == NULL
    assert act_grad(dy, dy) == ALIAS and act_grad(dy, dx, dx) == ALIAS
    half = dict(row_stride=200)
    assert act_grad(dy, rows(128 * MB, **half), rows(128 * MB + 100, **half)) == ALIAS     # 50 elements on, not 100
    assert act_grad(dy, rows(128 * MB, **half), rows(128 * MB + 202, **half)) == ALIAS     # reaches the next row's first
    assert act_grad(dy, rows(128 * MB, **half), rows(128 * MB + 200, row_stride=201)) == ALIAS
    # side by side: no alias, so that the next check's error is the one reported
    assert act_grad(dy, rows(128 * MB, **half), rows(128 * MB + 200, **half), up_steps=128 * MB) == ALIAS
    assert act_grad(dy, rows(128 * MB), rows(129 * MB, rows=3)) == BAD


def test_norm_arguments():
    x = rows()
    for eps in (0.0, -1.0, math.nan, math.inf, 2.0 ** -81, 2.0 ** 21):
        assert norm(x, eps=eps) == BAD
    assert norm(x, wtype=3) == BAD and norm(x, weight=5 * MB + 1) == MISALIGNED and norm(x, weight=5 * MB + 2, wtype=1) == MISALIGNED
    assert norm(x, inv=None) == NULL and norm(x, steps=None) == NULL and norm(x, inv=6 * MB + 2) == MISALIGNED
    assert norm(x, weight=128 * MB) == ALIAS and norm(x, inv=64 * MB) == ALIAS and norm(x, y=x) == ALIAS
    dy, dx = rows(), rows(128 * MB)
    assert norm_grad(dy, dx, inv=None) == NULL and norm_grad(dy, dx, ws=None) == NULL and norm_grad(dy, dx, codes=None) == NULL
    assert norm_grad(dy, dx, ws=8 * MB + 8) == MISALIGNED and norm_grad(dy, dx, gw=7 * MB + 1) == MISALIGNED
    assert norm_grad(dy, dy) == ALIAS and norm_grad(dy, dx, gw=5 * MB) == ALIAS and norm_grad(dy, dx, ws=7 * MB + 16 - 1600) == ALIAS
    assert norm_grad(dy, dx, wtype=7) == BAD and norm_grad(dy, rows(128 * MB, width=99)) == BAD
    assert norm_grad(dy, None, gw=None) == 0                        # nothing asked for
    assert fo.fo_rms_norm_workspace(10, 64) == 640 and fo.fo_rms_norm_workspace(10, 65) == 960
    assert fo.fo_rms_norm_workspace(10 ** 6, 64) == 1 << 22 and fo.fo_rms_norm_workspace(10 ** 6, 1 << 20) == 1 << 26
    assert fo.fo_rms_norm_workspace(10 ** 4, 16384) == 1 << 24 and fo.fo_rms_norm_workspace(10 ** 4, 32768) == 1 << 24
    assert fo.fo_rms_norm_workspace(0, 64) == 0


def test_rejected_calls_launch_nothing():
    before = fo.fo_kernel_launch_count()
    test_activation_arguments()
    test_norm_arguments()
    assert fo.fo_kernel_launch_count() == before


def test_python_refusals(monkeypatch):
    monkeypatch.setattr(fo, "_get_device", lambda: 0)
    x = torch.zeros(4, 64)
    for call in (A.compress, lambda t: A.activation(t, "silu"), A.rms_norm, lambda t: A.activation_forward(t, "swiglu")):
        with pytest.raises(ValueError, match="CUDA"):
            call(x)
    with pytest.raises(ValueError, match="kind"):
        A.activation(x, "relu")
    with pytest.raises(ValueError, match="kind"):
        A.activation(x, ["silu"])
    with pytest.raises(ValueError, match="second input"):
        A.activation(x, "gelu", up=x)
    with pytest.raises(ValueError, match="column"):
        A.compress(torch.zeros(()))
    with pytest.raises(ValueError, match="column"):
        A.rms_norm(torch.zeros(3, 0))
    with pytest.raises(TypeError, match="bfloat16"):
        A.compress(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(TypeError, match="one type"):
        A.linear(x, torch.zeros(3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="columns"):
        A.expand(A.Compressed(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.bfloat16), 64, torch.float32))
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, x)
        for call in (A.compress, lambda t: A.activation(t, "silu"), A.rms_norm, lambda t: A.linear(t, x)):
            with pytest.raises(NotImplementedError, match="tangent"):
                call(dual)


def fake(shape, stride, dtype=torch.bfloat16, device=0):
    """A CUDA tensor's description."""
    n = 1
    for s in shape:
        n *= s
    dense = stride == torch.empty(shape, device="meta").stride()
    return types.SimpleNamespace(shape=torch.Size(shape), stride=lambda: stride, is_contiguous=lambda: dense, dtype=dtype, is_cuda=True,
                                 device=types.SimpleNamespace(index=device), data_ptr=lambda: 4096, numel=lambda: n)


def test_layouts_of_rows(monkeypatch):
    monkeypatch.setattr(fo, "_get_device", lambda: 0)
    m = fo.matrix(fake((2, 3, 8), (24, 8, 1)))
    assert (m.rows, m.width, m.row_stride) == (6, 8, 8)
    m = fo.matrix(fake((2, 3, 8), (48, 16, 1)))
    assert (m.rows, m.row_stride) == (6, 16)
    assert fo.matrix(fake((2, 1, 8), (24, 8, 1))).row_stride == 24
    assert fo.matrix(fake((1, 3, 8), (0, 16, 1))).row_stride == 16
    assert fo.matrix(fake((8,), (1,))).rows == 1
    assert fo.matrix(fake((5, 8), (0, 1))).row_stride == 0
    assert fo.matrix(fake((5, 1), (7, 3))).row_stride == 7
    assert fo.matrix(fake((0, 3, 8), (24, 8, 1))).rows == 0 and fo.matrix(fake((3, 0, 8), (1, 8, 1))).rows == 0
    for bad in (fake((2, 3, 8), (32, 8, 1)), fake((5, 8), (1, 5)), fake((2, 3, 8), (8, 16, 1))):
        with pytest.raises(ValueError, match="contiguous"):
            fo.matrix(bad)
    with pytest.raises(ValueError, match="cuda:1"):
        fo.matrix(fake((5, 8), (8, 1), device=1))
    with pytest.raises(ValueError, match="rows of"):
        fo.matrix(fake((5, 8), (8, 1)), "up", fo.matrix(fake((5, 9), (9, 1))))


def test_reference_codes():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 0.4]])
    code, step = ref.codes(x)
    assert step.tolist() == [[1.0]] and code[0, :6].tolist() == [127, 0, 2, -2, 0, 0]
    x = torch.tensor([[-0.157226562]])
    code, step = ref.codes(x)
    assert step[0, 0] * 127 >= 0.157226562 > step[0, 0] * 127 * (1 - 2.0 ** -7) and code[0, 0] == -126
    x = torch.randn(64, 77, dtype=torch.float64).float()
    assert ((ref.kept(x) - x.double()).abs() <= ref.codes(x)[1].repeat_interleave(32, 1)[:, :77] * 0.5 * (1 + 2.0 ** -15)).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_reference_slopes_against_differences(kind):
    x = torch.linspace(-9, 9, 1801, dtype=torch.float64)
    h = 1e-5
    slope = (ref.act(kind, x + h)[0] - ref.act(kind, x - h)[0]) / (2 * h)
    # h^2 / 6 of a third derivative below 2, and 2^-52 of values below 10 over 2 h
    assert ((slope - ref.act(kind, x)[1]).abs() < 2 * h * h / 6 + 10 * 2.0 ** -52 / h).all()


def test_reference_norm_gradient_against_differences():
    torch.manual_seed(0)
    x = (torch.randint(-127, 128, (3, 32)) / 16).float()
    x[:, 0] = 127 / 16                                              # steps of 1/16: the codes stand for x itself
    assert torch.equal(ref.kept(x), x.double())
    w, dy = torch.randn(32), torch.randn(3, 32)
    grad, _, dw, _ = ref.norm_backward(x, w, 1e-5, dy)
    f = lambda x, w: (x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w * dy.double()).sum()
    x, w = x.double().requires_grad_(True), w.double().requires_grad_(True)
    gx, gw = torch.autograd.grad(f(x, w), (x, w))
    assert torch.allclose(gx, grad, atol=1e-12) and torch.allclose(gw, dw, atol=1e-12)
    h = 1e-5
    for i, j in ((0, 0), (1, 7), (2, 31)):
        d = torch.zeros(3, 32, dtype=torch.float64)
        d[i, j] = h
        assert abs(float((f(x + d, w) - f(x - d, w)) / (2 * h) - grad[i, j])) < 1e-6
