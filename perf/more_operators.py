"""Cases of the operators on activations kept in 8 bits for the backward pass, and of the policy loss on logits.

An activation is kept as int8 codes and one BF16 step for every 32 elements of a row (the last group of a row may be
partial). With a = max |x| of a group: step = the smallest BF16 number that is at least max(a / 127, 2^-126),
r = 1 / step rounded to 32 bits, code = x r (not rounded before) rounded to the nearest whole number, ties to even; the
element that a code stands for is x^ = code * step.

* checkpoint: x -> codes and steps -> x^ in x's type.
* activation: y = act(x), or act(gate) * up for the gated kinds (swiglu, geglu), whose input holds gate and up side by
  side in its last dimension; the gradient is taken at x^. "activation" makes the two calls itself,
  "activation_train" goes through automatic differentiation.
* norm: y = x r w, r = 1 / sqrt(mean x^2 + eps); with h = x^ r: dx = r (dy w - h mean(dy w h)), dw = sum over rows of dy h.
  "norm" and "norm_train" as above.
* policy: l = log softmax(x / T)[token], q = exp(l - old), loss = -min(q A, clip(q, 1 - lo, 1 + hi) A) +
  beta (exp(ref - l) - (ref - l) - 1), and its gradient. "policy_fused" gives weighted loss, l and gradient in one call,
  "policy_train" goes through automatic differentiation, "policy" is the loss alone. A negative token is no position:
  loss, l and gradient 0.

The sizes are those of this repository's GPT-2 small and Llama-3.1-8B tables (widths 768, 4096 and 14336, vocabularies
50257 and 128256), or generic.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
GROUP = 32
EPS = 1e-5
BYTES_MAX = 8192 * 128256 * 2 * 2      # of the largest listed case


def _rows(name, op, rows, width, dtype, kind="", wtype="", stride=0):
    c = dict(op=op, rows=rows, width=width, dtype=dtype, kind=kind, wtype=wtype or dtype, stride=stride)
    if name:
        c["name"] = name
    return c


def _policy(name, op, rows, vocab, dtype, lo=0.2, hi=0.2, beta=0.0, temperature=1.0, stride=0, pad_rows=0):
    c = dict(op=op, rows=rows, width=vocab, dtype=dtype, lo=lo, hi=hi, beta=beta, temperature=temperature, stride=stride,
             pad_rows=pad_rows)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token's hidden state: what a call costs at least
        _rows("checkpoint 1 token", "checkpoint", 1, 4096, "bf16"),
        # the input of a down projection over a batch of 32768 tokens
        _rows("checkpoint mlp", "checkpoint", 32768, 14336, "bf16"),
        # an odd width in 32 bits, rows in a wider buffer
        _rows("checkpoint odd f32", "checkpoint", 3001, 5003, "f32", stride=5010),
        # a gated MLP's activation in a training step of a few tokens
        _rows("swiglu few tokens", "activation", 16, 14336, "bf16", "swiglu"),
        # the same in a large step, under automatic differentiation
        _rows("swiglu training", "activation_train", 8192, 14336, "bf16", "swiglu"),
        # an odd width: rows of no common alignment
        _rows("geglu odd", "activation", 3001, 2731, "f16", "geglu"),
        # a norm before attention over a packed batch
        _rows("norm training", "norm_train", 16384, 4096, "bf16"),
        # GPT-2 small's width in 32 bits, one short sequence
        _rows("norm short f32", "norm", 128, 768, "f32"),
        # many short rows (a norm of each head's 128 elements), weight in 32 bits
        _rows("norm heads", "norm", 131072, 128, "bf16", wtype="f32"),
        # the smallest policy step: 16 sampled tokens
        _policy("policy step small", "policy_fused", 16, 50257, "bf16"),
        # one step of a large batch, a sixteenth of it padding, held near a reference model
        _policy("policy step large", "policy_fused", 8192, 128256, "bf16", hi=0.28, beta=0.04, pad_rows=512),
        # automatic differentiation, logits in 32 bits, odd vocabulary
        _policy("policy training f32", "policy_train", 1001, 50257, "f32", beta=0.1, temperature=0.8),
    ]


def draw(rng: random.Random):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    op = rng.choice(["checkpoint", "activation", "activation_train", "norm", "norm_train", "policy", "policy_fused",
                     "policy_fused", "policy_train"])
    while True:
        if op.startswith("policy"):
            rows, width = log(1, 16384), log(512, 262144)
            if rng.random() < 0.3:
                width = rng.choice([50257, 128256])
        else:
            rows, width = log(1, 65536), log(33, 16384)
            if rng.random() < 0.5:             # widths of models are multiples of 64
                width = max(64, width // 64 * 64)
        c = _policy("", op, rows, width, dtype, lo=rng.choice([0.2, round(rng.uniform(0.05, 0.3), 3)]),
                    hi=rng.choice([0.2, round(rng.uniform(0.05, 0.5), 3)]),
                    beta=rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.2), 3)]),
                    temperature=rng.choice([1.0, round(rng.uniform(0.5, 2.0), 2)]),
                    stride=rng.choice([0, 0, width + rng.randint(1, 100)]),
                    pad_rows=rng.choice([0, rows // 10])) if op.startswith("policy") else \
            _rows("", op, rows, width, dtype, rng.choice(["silu", "gelu", "swiglu", "geglu"]) if "act" in op else "",
                  wtype=rng.choice([dtype, "f32"]) if op.startswith("norm") else "",
                  stride=rng.choice([0, 0, 0, 1]) if op == "checkpoint" else 0)
        if c["stride"] == 1:
            c["stride"] = width + rng.randint(1, 64)
        if work(c)["bytes"] <= BYTES_MAX:
            return c


def _gated(case):
    return case.get("kind") in ("swiglu", "geglu")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, w, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
    randn = lambda *size, dtype=torch.float32: torch.randn(size, generator=g, device="cuda", dtype=dtype)
    rand = lambda *size: torch.rand(size, generator=g, device="cuda")
    if case["op"].startswith("policy"):
        return _prepare_policy(case, n, w, dt, randn, rand)
    cols = 2 * w if _gated(case) else w
    x = randn(n, max(case["stride"], cols), dtype=dt)[:, :cols]
    # channels differ in size, a few of them by much
    channel = torch.exp(0.5 * randn(cols)) * torch.where(rand(cols) < 0.004, 20.0, 1.0)
    x.mul_(channel.to(dt))
    s = dict(case=case, x=x)
    if case["op"] != "checkpoint":
        s["grad"] = randn(n, w, dtype=dt).mul_(0.01)
    if case["op"].startswith("norm"):
        s["weight"] = (1 + 0.1 * randn(w)).to(DTYPES[case["wtype"]])
    return s


def _prepare_policy(case, n, v, dt, randn, rand):
    x = randn(n, case["stride"] or v, dtype=dt)[:, :v].mul_(2.5)
    # a few plausible tokens at each position, one of them sampled
    ids = ((rand(n, 1) * v).long() + ((rand(n, 1) * (v // 8 - 1)).long() + 1) * torch.arange(8, device="cuda")) % v
    x.scatter_add_(1, ids, (torch.linspace(10.0, 0.0, 8, device="cuda") + rand(n, 8)).to(dt))
    tokens = ids.gather(1, (rand(n, 1) ** 2 * 8).long().clamp_(max=7))[:, 0].contiguous()
    block = max(1, 2 ** 27 // v)
    lse = torch.cat([torch.logsumexp(x[i:i + block].float() / case["temperature"], 1) for i in range(0, n, block)])
    logp = x.gather(1, tokens[:, None])[:, 0].float() / case["temperature"] - lse
    # the policy has moved since it sampled: ratios around 1, a third of them clipped, none on the very border
    moved = 0.25 * randn(n)
    for border in (math.log(1 - case["lo"]), math.log(1 + case["hi"])):
        moved = torch.where((moved - border).abs() < 1e-3, moved + 4e-3, moved)
    s = dict(case=case, x=x, tokens=tokens, old=logp - moved, advantage=randn(n),
             ref=logp + 0.2 * randn(n) if case["beta"] else None, weight=(0.5 + rand(n)) / n)
    if case["pad_rows"]:
        tokens[n - case["pad_rows"]:] = -1
        s["weight"][n - case["pad_rows"]:] = 0.0
    return s


# --- the plain form: 32-bit elementary operations --------------------------------------------------------------------

def _plain_kept(x):
    """What the codes of x stand for, in 32 bits."""
    n, w = x.shape
    groups = -(-w // GROUP)
    y = torch.zeros((n, groups * GROUP), device=x.device)
    y[:, :w] = x
    y = y.view(n, groups, GROUP)
    a = y.abs().amax(2, keepdim=True)
    cut = ((a / 127).clamp(min=2.0 ** -126).view(torch.int32) & -65536)
    step = torch.where(cut.view(torch.float32) * 127 < a, cut + 65536, cut).view(torch.float32)
    # the product in 64 bits: next to a half, 32 would round it to the half itself
    code = torch.round(y.double() * (1 / step).double()).float()
    return (code * step).view(n, groups * GROUP)[:, :w]


def _plain_act(kind, x):
    """act and its derivative."""
    if kind in ("silu", "swiglu"):
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    cdf = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
    return x * cdf, cdf + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))


def _plain_activation(s):
    case, dt = s["case"], s["x"].dtype
    x, dy = s["x"].float(), s["grad"].float()
    if not _gated(case):
        kept = _plain_kept(x)
        return {"y": _plain_act(case["kind"], x)[0].to(dt), "grad": (dy * _plain_act(case["kind"], kept)[1]).to(dt)}
    w = case["width"]
    y = _plain_act(case["kind"], x[:, :w])[0] * x[:, w:]
    gate, up = _plain_kept(x[:, :w]), _plain_kept(x[:, w:])
    f, d = _plain_act(case["kind"], gate)
    return {"y": y.to(dt), "grad": torch.cat([dy * up * d, dy * f], 1).to(dt)}


def _plain_norm(s):
    x, dy, w = s["x"].float(), s["grad"].float(), s["weight"].float()
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    h = _plain_kept(x) * r
    g = dy * w
    dx = r * (g - h * (g * h).mean(1, keepdim=True))
    return {"y": (x * r * w).to(s["x"].dtype), "grad": dx.to(s["x"].dtype),
            "grad_weight": (dy * h).sum(0, dtype=torch.float64).to(s["weight"].dtype)}


def _plain_policy(s):
    case = s["case"]
    there = s["tokens"] >= 0
    t = s["tokens"].clamp(min=0)[:, None]
    d = s["x"].float() / case["temperature"]
    d = d - d.amax(1, keepdim=True)
    e = d.exp()
    z = e.sum(1, keepdim=True)
    logp = (d.gather(1, t) - z.log())[:, 0]
    q, a = torch.exp(logp - s["old"]), s["advantage"]
    clipped = q.clamp(1 - case["lo"], 1 + case["hi"])
    loss = -torch.minimum(q * a, clipped * a)
    c = -a * q * torch.where(a >= 0, q <= 1 + case["hi"], q >= 1 - case["lo"])
    if s["ref"] is not None:
        k = s["ref"] - logp
        loss = loss + case["beta"] * (torch.exp(k) - k - 1)
        c = c + case["beta"] * (1 - torch.exp(k))
    zero = torch.zeros_like(loss)
    loss, c, logp = torch.where(there, loss, zero), torch.where(there, c, zero), torch.where(there, logp, zero)
    if case["op"] == "policy":
        return {"loss": loss, "logp": logp}
    c = (c * s["weight"] / case["temperature"])[:, None]
    grad = (e * (-c / z)).scatter_add_(1, t, c).to(s["x"].dtype)
    return {"loss": loss * s["weight"] if case["op"] == "policy_fused" else loss, "logp": logp, "grad": grad}


# --- the framework's operators ----------------------------------------------------------------------------------------

def _own(s):
    case, x, op = s["case"], s["x"], s["case"]["op"]
    if op.startswith("policy"):
        from quantized_optimizer_state_gb300 import losses
        how = dict(clip_low=case["lo"], clip_high=case["hi"], ref_logp=s["ref"], kl_weight=case["beta"],
                   temperature=case["temperature"])
        if op == "policy_fused":
            o = losses.policy_loss_grad(x, s["tokens"], s["old"], s["advantage"], row_weight=s["weight"], **how)
            return {"loss": o.loss, "logp": o.logp, "grad": o.grad}
        if op == "policy":
            o = losses.policy_loss(x, s["tokens"], s["old"], s["advantage"], **how)
            return {"loss": o.loss, "logp": o.logp}
        x = x.detach().requires_grad_(True)
        o = losses.policy_loss(x, s["tokens"], s["old"], s["advantage"], **how)
        grad, = torch.autograd.grad(o.loss, x, s["weight"])
        return {"loss": o.loss.detach(), "logp": o.logp, "grad": grad}
    from quantized_optimizer_state_gb300 import activations
    if op == "checkpoint":
        return {"x": activations.expand(activations.compress(x))}
    if op == "activation":
        y, kept = activations.activation_forward(x, case["kind"])
        return {"y": y, "grad": activations.activation_backward(kept, s["grad"])}
    if op == "norm":
        y, kept = activations.rms_norm_forward(x, s["weight"], eps=EPS)
        grad, grad_weight = activations.rms_norm_backward(kept, s["grad"])
        return {"y": y, "grad": grad, "grad_weight": grad_weight}
    x = x.detach().requires_grad_(True)
    if op == "activation_train":
        y = activations.activation(x, case["kind"])
        grad, = torch.autograd.grad(y, x, s["grad"])
        return {"y": y.detach(), "grad": grad}
    w = s["weight"].detach().requires_grad_(True)
    y = activations.rms_norm(x, w, eps=EPS)
    grad, grad_weight = torch.autograd.grad(y, (x, w), s["grad"])
    return {"y": y.detach(), "grad": grad, "grad_weight": grad_weight}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    with torch.no_grad():
        if op == "checkpoint":
            return {"x": _plain_kept(state["x"].float()).to(state["x"].dtype)}
        if op.startswith("activation"):
            return _plain_activation(state)
        return _plain_norm(state) if op.startswith("norm") else _plain_policy(state)


def work(case):
    n, w, b, op = case["rows"], case["width"], BYTES[case["dtype"]], case["op"]
    if op.startswith("policy"):
        small = n * (28 + 4 * bool(case["beta"]))
        read = (n - case["pad_rows"]) * w * b
        return {"bytes": read + small + (0 if op == "policy" else n * w * b), "flops": n * w * (4 if op == "policy" else 8)}
    kept = n * (w + 2 * -(-w // GROUP))
    if op == "checkpoint":
        return {"bytes": 2 * (n * w * b + kept), "flops": n * w * 5}
    if op.startswith("norm"):
        return {"bytes": 4 * n * w * b + 2 * kept + 8 * n + 3 * w * BYTES[case["wtype"]], "flops": n * w * 17}
    parts = 2 if _gated(case) else 1
    # read x, write y and the codes; read dy and the codes, write dx
    return {"bytes": n * w * b * (2 + 2 * parts) + 2 * parts * kept, "flops": n * w * (16 + 8 * parts)}


# --- 64 bits, from the definitions ------------------------------------------------------------------------------------

def _exact_kept(x):
    """x^ from 64-bit x [n, w]."""
    parts = []
    for i in range(0, x.shape[1], 32 * 512):
        piece = x[:, i:i + 32 * 512]
        n, w = piece.shape
        y = torch.nn.functional.pad(piece, (0, -w % 32)).reshape(n, -1, 32)
        mantissa, exponent = torch.frexp((y.abs().max(2).values / 127).clamp(min=2.0 ** -126))
        step = torch.ldexp(torch.ceil(mantissa * 256) / 256, exponent).float().double()   # undoes a rounding of the power
        r = (1 / step).float().double()
        parts.append((torch.round(y * r[:, :, None]) * step[:, :, None]).reshape(n, -1)[:, :w])
    return torch.cat(parts, 1)


def _exact_act(kind, x):
    if kind in ("silu", "swiglu"):
        s = torch.sigmoid(x)
        return x * s, s + x * s * torch.sigmoid(-x)
    cdf = 0.5 * torch.erfc(-x / math.sqrt(2))
    return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


def _exact_block(s, i, j):
    case = s["case"]
    op, x = case["op"], s["x"][i:j].double()
    if op == "checkpoint":
        return {"x": _exact_kept(x)}
    if op.startswith("activation"):
        dy = s["grad"][i:j].double()
        if not _gated(case):
            return {"y": _exact_act(case["kind"], x)[0], "grad": dy * _exact_act(case["kind"], _exact_kept(x))[1]}
        gate, up = x.chunk(2, 1)
        f, d = _exact_act(case["kind"], _exact_kept(gate))
        return {"y": _exact_act(case["kind"], gate)[0] * up, "grad": torch.cat([dy * _exact_kept(up) * d, dy * f], 1)}
    if op.startswith("norm"):
        dy, w = s["grad"][i:j].double(), s["weight"].double()
        rms = torch.sqrt((x ** 2).mean(1, keepdim=True) + EPS)
        h = _exact_kept(x) / rms
        return {"y": x / rms * w, "grad": (dy * w - h * (dy * w * h).mean(1, keepdim=True)) / rms,
                "grad_weight": (dy * h).sum(0)}
    t, a, old = s["tokens"][i:j], s["advantage"][i:j].double(), s["old"][i:j].double()
    there = t >= 0
    logp = torch.log_softmax(x / case["temperature"], 1)
    l = logp.gather(1, t.clamp(min=0)[:, None])[:, 0]
    ratio = (l - old).exp()
    bound = torch.where(a >= 0, torch.minimum(ratio, torch.full_like(ratio, 1 + case["hi"])),
                        torch.maximum(ratio, torch.full_like(ratio, 1 - case["lo"])))
    loss, slope = -a * bound, torch.where(bound == ratio, -a * ratio, 0.0)
    if s["ref"] is not None:
        k = s["ref"][i:j].double() - l
        loss, slope = loss + case["beta"] * (torch.expm1(k) - k), slope - case["beta"] * torch.expm1(k)
    loss, slope, l = [torch.where(there, v, 0.0) for v in (loss, slope, l)]
    if op == "policy":
        return {"loss": loss, "logp": l}
    w = s["weight"][i:j].double()
    p = -logp.exp()
    p[torch.arange(j - i, device=x.device), t.clamp(min=0)] += 1
    return {"loss": loss * w if op == "policy_fused" else loss, "logp": l,
            "grad": p * (slope * w / case["temperature"])[:, None]}


def exact(case, seed):
    s = prepare(case, seed)
    n = case["rows"]
    block = max(1, 2 ** 26 // s["x"].shape[1])
    with torch.no_grad():
        parts = [_exact_block(s, i, min(i + block, n)) for i in range(0, n, block)]
        return {key: sum(p[key] for p in parts) if key == "grad_weight" else torch.cat([p[key] for p in parts])
                for key in parts[0]}
