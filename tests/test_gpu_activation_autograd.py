"""Operators on activations as a training step uses them: automatic differentiation, all together, in graphs, on
streams and threads, and what stands around their outputs."""
import math
import threading

import pytest
import torch

from quantized_optimizer_state_gb300 import activations as A
from quantized_optimizer_state_gb300 import fo
from quantized_optimizer_state_gb300.losses import policy_loss_grad
from tests import act_reference as ref
from tests.test_gpu_activations import halves, make, same
from tests.test_gpu_loss_guards import Guarded

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fo.lib()


@pytest.mark.parametrize("kind", list(A.KINDS))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd_gives_what_the_pairs_give(kind, dtype):
    gated = kind in ("swiglu", "geglu")
    x, dy = make((2, 5, 2 * 72 if gated else 72), dtype), make((2, 5, 72), dtype, seed=1)
    y0, kept = A.activation_forward(x, kind)
    want = A.activation_backward(kept, dy)
    leaf = x.clone().requires_grad_(True)
    y = A.activation(leaf, kind)
    assert torch.equal(y, y0)
    y.backward(dy)
    assert torch.equal(leaf.grad, want) and leaf.grad.shape == x.shape
    if gated:
        a, b = (t.contiguous().requires_grad_(True) for t in halves(x))
        A.activation(a, kind, up=b).backward(dy)
        assert torch.equal(torch.cat([a.grad, b.grad], -1), want)
        (c,) = torch.autograd.grad(A.activation(a.detach(), kind, up=b), b, dy)      # one of the two
        assert torch.equal(c, b.grad)
        twice = a.detach().clone().requires_grad_(True)                             # the same tensor as both
        A.activation(twice, kind, up=twice).backward(dy)
        ya, ka = A.activation_forward(twice.detach(), kind, up=twice.detach())
        g, u = A.activation_backward(ka, dy)
        assert torch.equal(twice.grad, g + u)
    A.activation(leaf, kind).sum().backward()                                       # an expanded incoming gradient
    with torch.no_grad():
        assert torch.equal(A.activation(leaf, kind), y0) and not A.activation(leaf, kind).requires_grad


@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (BF, F32), (F32, F32)])
def test_norm_autograd(dtype, wtype):
    x, dy = make((4, 6, 200), dtype), make((4, 6, 200), dtype, seed=1)
    weight = (1 + make((200,), F32, seed=2, scale=0.1)).to(wtype)
    y0, kept = A.rms_norm_forward(x, weight)
    gx, gw = A.rms_norm_backward(kept, dy)
    a, w = x.clone().requires_grad_(True), weight.clone().requires_grad_(True)
    A.rms_norm(a, w).backward(dy)
    assert torch.equal(a.grad, gx) and torch.equal(w.grad, gw)
    assert torch.equal(torch.autograd.grad(A.rms_norm(a, weight), a, dy)[0], gx)
    assert torch.equal(torch.autograd.grad(A.rms_norm(x, w), w, dy)[0], gw)
    free, = torch.autograd.grad(A.rms_norm(a), a, dy)
    assert torch.equal(free, A.rms_norm_backward(A.rms_norm_forward(x)[1], dy)[0])
    y = A.rms_norm(a, w)
    with torch.no_grad():
        w.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified"):                             # the weight that the gradient needs
        y.backward(dy)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear(dtype):
    x, w, b = make((3, 7, 100), dtype), make((60, 100), dtype, seed=1, scale=0.1), make((60,), dtype, seed=2)
    dy = make((3, 7, 60), dtype, seed=3)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = A.linear(*leaves)
    assert torch.equal(y, torch.nn.functional.linear(x, w, b))
    y.backward(dy)
    d, xh = dy.double().reshape(-1, 60), A.expand(A.compress(x)).double().reshape(-1, 100)
    # sums of 60 or 21 products: their roundings, and the one to the type
    tol = 64 * 2.0 ** -24
    ref.close(leaves[0].grad.reshape(-1, 100), d @ w.double(), d.abs() @ w.double().abs() * tol, "gradient of x")
    ref.close(leaves[1].grad, d.t() @ xh, d.abs().t() @ xh.abs() * tol, "gradient of the weight")
    ref.close(leaves[2].grad, d.sum(0), d.abs().sum(0) * tol, "gradient of the bias")
    only, = torch.autograd.grad(A.linear(leaves[0], w), leaves[0], dy)
    assert torch.equal(only, leaves[0].grad)
    with torch.autocast("cuda", dtype=BF):
        inside = A.linear(leaves[0], leaves[1])
        assert inside.dtype == dtype
    inside.backward(dy)


def test_a_block_op_by_op():
    """norm, product, gated activation, product: each op's gradient is its formula's at what it kept, for the gradient
    that reached it."""
    torch.manual_seed(0)
    n, d, f = 96, 160, 112
    h = make((n, d), BF).requires_grad_(True)
    wn = (1 + make((d,), F32, seed=1, scale=0.1)).to(BF).requires_grad_(True)
    w1, w2 = (make(s, BF, seed=i, scale=0.05).requires_grad_(True) for i, s in ((2, (2 * f, d)), (3, (d, f))))
    seen = {}

    def watch(name, t):
        t.register_hook(lambda g: seen.__setitem__(name, g))
        return t

    x = watch("x", A.rms_norm(h, wn, eps=1e-5))
    gu = watch("gu", A.linear(x, w1))
    a = watch("a", A.activation(gu, "swiglu"))
    y = watch("y", A.linear(a, w2))
    (y.float() ** 2).sum().backward()
    grad, tol, dw, dw_tol = ref.norm_backward(h.detach(), wn.detach(), 1e-5, seen["x"])
    ref.close(h.grad, grad, tol, "norm")
    ref.close(wn.grad, dw, dw_tol, "norm's weight")
    g, gt, u, ut = ref.backward("swiglu", halves(gu.detach())[0], seen["a"], halves(gu.detach())[1])
    ref.close(seen["gu"], torch.cat([g, u], 1), torch.cat([gt, ut], 1), "gated activation")
    for w, inp, out in ((w1, x, "gu"), (w2, a, "y")):
        dy, kept = seen[out].double(), A.expand(A.compress(inp.detach())).double()
        ref.close(w.grad, dy.t() @ kept, dy.abs().t() @ kept.abs() * 128 * 2.0 ** -24, "weight")


def test_gradients_against_differences():
    """Inputs that their codes stand for exactly: the gradient is that of the forward pass itself."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randint(-127, 128, (3, 64), generator=g, device="cuda").float() / 32
    x[:, ::32] = 127 / 32
    assert torch.equal(A.expand(A.compress(x)), x)
    dy, other = make((3, 64), F32, seed=1), x.flip(0).contiguous()
    h = 2.0 ** -6
    for f in (lambda t: A.activation(t, "silu"), lambda t: A.activation(t, "gelu"), lambda t: A.rms_norm(t, eps=1e-3),
              lambda t: A.activation(t, "swiglu", up=other), lambda t: A.activation(other, "geglu", up=t)):
        leaf = x.clone().requires_grad_(True)
        grad, = torch.autograd.grad(f(leaf), leaf, dy)
        for i, j in ((0, 1), (1, 33), (2, 63), (2, 0)):
            d = torch.zeros_like(x)
            d[i, j] = h
            up, down = ((f(x + s * d).double() * dy.double()).sum() for s in (1, -1))
            # h^2 / 6 of a third derivative below 2 |dy up|, and the roundings of 64 results over 2 h
            size = float(dy.abs().max()) * 5
            assert abs(float((up - down) / (2 * h) - grad[i, j])) <= size * (2 * h * h / 6 + 64 * 2.0 ** -23 / h)


def test_second_derivatives_are_refused():
    x = make((4, 64), F32).requires_grad_(True)
    for f in (lambda t: A.activation(t, "silu"), A.rms_norm):
        g, = torch.autograd.grad(f(x).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()


def step(x, dy, w, dyn):
    y, kept = A.activation_forward(x, "swiglu")
    z, kept_norm = A.rms_norm_forward(y, w)
    back = A.expand(A.compress(z))
    gy, gw = A.rms_norm_backward(kept_norm, dyn)
    return y, z, back, gy, gw, A.activation_backward(kept, dy)


def inputs(seed, n=500, f=328, dtype=BF):
    return (make((n, 2 * f), dtype, seed=seed), make((n, f), dtype, seed=seed + 1), 1 + make((f,), F32, seed=seed + 2, scale=0.1),
            make((n, f), dtype, seed=seed + 3))


def test_captured_and_replayed():
    args = [t.clone() for t in inputs(0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*args)
        leaf = args[0].clone().requires_grad_(True)
        torch.autograd.grad(A.activation(leaf, "swiglu"), leaf, args[1])
    torch.cuda.current_stream().wait_stream(side)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        first = step(*args)
    leaf = args[0].detach().requires_grad_(True)
    with torch.cuda.graph(two):                                    # another graph with temporaries of its own
        second = step(*args)
        grad, = torch.autograd.grad(A.activation(leaf, "swiglu"), leaf, args[1])
    for seed in (5, 6):
        for t, new in zip(args, inputs(seed)):
            t.copy_(new)
        one.replay()
        two.replay()
        one.replay()
        torch.cuda.synchronize()
        want = step(*inputs(seed))
        assert all(torch.equal(p, q) for p, q in zip(first, want)) and all(torch.equal(p, q) for p, q in zip(second, want))
        assert torch.equal(grad, want[-1])


def test_policy_captured_and_replayed():
    from tests.test_gpu_policy import make as sampled
    x, t, old, a, r, w = sampled(300, 5003, BF, seed=1)
    how = dict(ref_logp=r, kl_weight=0.1, row_weight=w)
    want = policy_loss_grad(x, t, old, a, **how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = policy_loss_grad(x, t, old, a, **how)
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    x2, t2, old2, a2, r2, w2 = sampled(300, 5003, BF, seed=2)
    for p, q in ((x, x2), (t, t2), (old, old2), (a, a2), (r, r2), (w, w2)):
        p.copy_(q)
    graph.replay()
    want = policy_loss_grad(x2, t2, old2, a2, ref_logp=r2, kl_weight=0.1, row_weight=w2)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_streams_and_threads():
    """Calls of several host threads, each on a stream of its own."""
    cases = [inputs(10 * i, n=300 + 50 * i, f=[328, 64, 777, 4096][i]) for i in range(4)]
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step(*cases[i])
            stream.synchronize()
            if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                wrong.append(i)
        except Exception as e:                                     # noqa: BLE001 - reported by the main thread
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cut", [0, 1, 2, 3])
@pytest.mark.parametrize("n,w", [(1, 1), (3, 33), (5, 64), (700, 40), (9, 4096), (4, 5001)])
def test_what_stands_around(n, w, cut, dtype):
    """Nothing is written before or after any output, at every alignment of the matrices."""
    g = fo.groups(w)
    x, up, dy = (make((n, w), dtype, seed=i) + 0.25 for i in range(3))
    kept = [Guarded(n * g * 32, torch.int16, 0) for _ in range(2)]          # marks are 16-bit numbers: codes by view
    code_bytes = [torch.full((128 + n * g * 32 + 128,), 77, dtype=torch.int8, device="cuda") for _ in range(2)]
    codes = [b[128:128 + n * g * 32].view(n, g * 32) for b in code_bytes]
    steps = [Guarded(n * g, BF, cut) for _ in range(2)]
    y = Guarded(n * w, dtype, cut)
    at = lambda a: a.of.view(n, w)
    fo.fo_activation(0, x, at(y), codes[0], steps[0].of.view(n, g), up, codes[1], steps[1].of.view(n, g))
    y.check("y")
    grads = [Guarded(n * w, dtype, cut) for _ in range(2)]
    fo.fo_activation_grad(0, codes[0], steps[0].of, dy, at(grads[0]), codes[1], steps[1].of, at(grads[1]))
    for a in grads:
        a.check("gradient")
    out, inv, gx, gw = Guarded(n * w, dtype, cut), Guarded(n, F32, cut), Guarded(n * w, dtype, cut), Guarded(w, F32, cut)
    ws = Guarded(fo.fo_rms_norm_workspace(n, w), F32, 0)
    weight = make((w,), F32, seed=9)
    fo.fo_rms_norm(x, at(out), weight, 1e-6, inv.of, codes[0], steps[0].of)
    fo.fo_rms_norm_grad(codes[0], steps[0].of, inv.of, dy, at(gx), weight, gw.of, ws.of)
    for name, a in (("norm", out), ("inverse rms", inv), ("gradient", gx), ("weight's gradient", gw)):
        a.check(name)
    assert (ws.all[:ws.lo] == ws.mark).all() and (ws.all[ws.hi:] == ws.mark).all()
    back = Guarded(n * w, dtype, cut)
    fo.fo_compress(x, codes[1], steps[1].of)
    fo.fo_expand(codes[1], steps[1].of, at(back))
    back.check("expanded")
    for b in code_bytes:
        assert (b[:128] == 77).all() and (b[-128:] == 77).all()
    for s in steps:
        s.check("steps")
    del kept


def test_one_library_in_the_process():
    """The PyTorch module and the ctypes binding call the same library: one counts the other's launches."""
    x, before = make((4, 64), F32), fo.fo_kernel_launch_count()
    c = A.compress(x)
    assert fo.fo_kernel_launch_count() == before + 1
    fo.fo_expand(c.codes, c.steps, x)
    A.rms_norm_backward(A.rms_norm_forward(x, torch.ones(64, device="cuda"))[1], x)
    assert fo.fo_kernel_launch_count() == before + 5


def test_outputs_count_as_modified():
    x = make((4, 64), F32).requires_grad_(True)
    out = torch.empty(4, 64, device="cuda")
    c = A.compress(x.detach())
    y = out * x                                                    # saves out
    A.expand(c, out=out)
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


def test_refusals_on_the_device():
    x = make((4, 64), BF)
    y, kept = A.activation_forward(x, "swiglu")
    with pytest.raises(ValueError, match="shape"):
        A.activation_backward(kept, x)
    with pytest.raises(ValueError, match="float32"):
        A.activation_backward(kept, y.float())
    with pytest.raises(ValueError, match="even"):
        A.activation(x[:, :63], "swiglu")
    with pytest.raises(ValueError, match="gate's shape"):
        A.activation(x, "swiglu", up=x[:2])
    with pytest.raises(ValueError, match="type"):
        A.activation(x, "swiglu", up=x.float())
    with pytest.raises(ValueError, match="contiguous"):
        A.compress(x.t())
    with pytest.raises(ValueError, match="weight"):
        A.rms_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError, match="weight"):
        A.rms_norm(x, torch.ones(64, dtype=torch.float64, device="cuda"))
    with pytest.raises(fo.FoError):
        A.rms_norm(x, eps=0.0)
    with pytest.raises(ValueError, match="out"):
        A.expand(A.compress(x), out=x[:2])
    with pytest.raises(TypeError, match="codes"):
        fo.fo_expand(torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), A.compress(x).steps, x)
    with pytest.raises(ValueError, match="steps holds"):
        fo.fo_expand(torch.zeros(4, 64, dtype=torch.int8, device="cuda"), A.compress(x).steps[:2], x)


def test_example_runs_and_its_gradients_are_near_those_of_full_precision():
    """The example trains; the gradients of its model, whose activations are kept in 8 bits, are those of the same
    model in 64 bits up to the roundings of 16-bit activations and of the codes."""
    from quantized_optimizer_state_gb300 import policy_example as ex
    r = ex.run(vocab=211, dim=64, hidden=88, blocks=2, contexts=8, samples=8, steps=3)
    assert len(r["rewards"]) == 3 and all(math.isfinite(v) for v in r["rewards"] + r["losses"])
    torch.manual_seed(3)
    model = ex.Policy(211, 64, 88, 2, "cuda")                      # FP32: what is left are the codes
    tokens = torch.arange(40, device="cuda") % 211
    dy = torch.randn(40, 211, device="cuda") * 0.01
    model(tokens).backward(dy)

    def plain(m):
        p = {k: v.detach().double().requires_grad_(True) for k, v in m.named_parameters()}
        norm = lambda h, w: h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w
        h = p["embed.weight"][tokens]
        for i in range(2):
            gate, up = (norm(h, p[f"blocks.{i}.norm"]) @ p[f"blocks.{i}.gate_up"].t()).chunk(2, 1)
            h = h + (torch.nn.functional.silu(gate) * up) @ p[f"blocks.{i}.down"].t()
        (norm(h, p["norm"]) @ p["head"].t()).backward(dy.double())
        return {k: v.grad for k, v in p.items()}

    for name, want in plain(model).items():
        got = dict(model.named_parameters())[name].grad.double()
        # a code is within 1/254 of its group's largest, some 0.5 % of an element's typical size, at up to seven places on
        # the way; what is checked is that nothing is missing or transposed
        assert float((got - want).norm() / want.norm()) < 7 * 0.01, name
