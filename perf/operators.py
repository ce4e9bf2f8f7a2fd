"""Cases of the loss operators: log probabilities of given tokens (with entropy and top alternatives) and
distillation from a teacher's top logits, each forward and backward.

Notation: x the logits of one row, T the temperature, s = x / T, m = max s, Z = sum exp(s - m), p = exp(s - m) / Z.

* logprobs: log p[token], H = -sum p log p, the ids and log probabilities of the K most probable tokens
  (ties go to the lowest id).
* logprobs_train: log p[token] and H, and the gradient of sum g log p[token] + h H for given g and h by row.
* distill, distill_train, distill_fused: KL(q || p) for a teacher q known by K ids and logits. q is renormalised over
  the K, or (tail) the rest of both distributions is one more outcome. "distill" gives the loss by row,
  "distill_train" the loss and then the gradient for a given weight by row (two calls, as automatic
  differentiation makes them), "distill_fused" weighted loss and gradient in one call.

The vocabularies 50257 and 128256 are those of this repository's GPT-2 small and Llama-3.1-8B tables.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
VOCAB_MAX = 262144
WORK_MAX = 8192 * 128256 * 4          # bytes of the largest listed case (logits read, gradient written)


def _case(name, op, rows, vocab, dtype, k=0, temperature=1.0, pad=0, stride=0, tail=False, short=False, masked_rows=0):
    c = dict(op=op, rows=rows, vocab=vocab, dtype=dtype, k=k, temperature=temperature, pad=pad, stride=stride,
             tail=tail, short=short, masked_rows=masked_rows)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token of one sequence while serving, with the five alternatives that an API answers with
        _case("logprobs 1 token", "logprobs", 1, 128256, "bf16", k=5),
        # a step of 64 sequences whose logits the head left in 32 bits, 20 alternatives, sampling temperature
        _case("logprobs 64 f32", "logprobs", 64, 128256, "f32", k=20, temperature=0.8),
        # scoring a long prompt: no alternatives
        _case("logprobs score", "logprobs", 4096, 128256, "bf16"),
        # writing down a teacher's answers: 64 alternatives a position, odd vocabulary, rows of no common alignment
        _case("logprobs teacher", "logprobs", 3001, 50257, "bf16", k=64),
        # policy training on sampled tokens: log probabilities, entropy, and both gradients
        _case("logprobs train", "logprobs_train", 4096, 128256, "bf16", temperature=0.7),
        # the same in 32 bits on a short odd batch, rows padded to a multiple of 64, unused ids masked
        _case("logprobs train f32", "logprobs_train", 333, 50257, "f32", pad=57, stride=50304),
        # evaluation of a student: loss alone
        _case("distill eval", "distill", 2048, 50257, "f16", k=32, temperature=2.0),
        # a student under automatic differentiation: loss, then its gradient
        _case("distill autograd", "distill_train", 2048, 128256, "bf16", k=64, temperature=2.0),
        # the smallest training step: a few rows
        _case("distill step small", "distill_fused", 16, 50257, "bf16", k=8),
        # one training step of a large batch, a sixteenth of it padding
        _case("distill step large", "distill_fused", 8192, 128256, "bf16", k=64, temperature=1.5, masked_rows=512),
        # the rest of the vocabulary as one outcome, in 32 bits, answers of unequal length
        _case("distill step tail f32", "distill_fused", 1001, 128256, "f32", k=20, tail=True, short=True),
        # GPT-2 small's batch: 8 sequences of 1024, odd vocabulary, 100 ids with a tail
        _case("distill step gpt2", "distill_fused", 8192, 50257, "bf16", k=100, tail=True),
    ]


def draw(rng: random.Random):
    op = rng.choice(["logprobs", "logprobs", "logprobs_train", "distill", "distill_train", "distill_fused", "distill_fused"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    while True:
        rows, vocab = log(1, 16384), log(512, VOCAB_MAX)
        if rng.random() < 0.3:
            vocab = rng.choice([50257, 128256])
        if rows * vocab * BYTES[dtype] * 2 <= WORK_MAX:
            break
    k = rng.choice([0, log(1, 128)]) if op == "logprobs" else 0 if op == "logprobs_train" else log(1, 128)
    distill = op.startswith("distill")
    return _case("", op, rows, vocab, dtype, k=k, temperature=rng.choice([1.0, round(rng.uniform(0.5, 4.0), 2)]),
                 pad=rng.choice([0, 0, rng.randint(1, vocab // 8)]),
                 stride=rng.choice([0, 0, vocab + rng.randint(1, 100)]),
                 tail=distill and rng.random() < 0.5, short=distill and rng.random() < 0.3,
                 masked_rows=rng.choice([0, rows // 10]) if op == "distill_fused" else 0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, v, k, dt = case["rows"], case["vocab"], case["k"], DTYPES[case["dtype"]]
    rand = lambda *size: torch.rand(size, generator=g, device="cuda")
    live = v - case["pad"]                        # ids from `live` on are no tokens: masked
    x = torch.randn((n, case["stride"] or v), generator=g, device="cuda", dtype=dt)[:, :v].mul_(2.5)
    # the next token's few plausible candidates, spread over the vocabulary without repetition
    kk = max(k, 8)
    step = (rand(n, 1) * (live // kk - 1)).long() + 1
    ids = ((rand(n, 1) * live).long() + step * torch.arange(kk, device="cuda")) % live
    lift = torch.linspace(10.0, 0.0, kk, device="cuda") + rand(n, kk)
    x.scatter_add_(1, ids, lift.to(dt))
    if case["pad"]:
        x[:, live:] = -math.inf
    s = dict(case=case, x=x)
    if case["op"].startswith("logprobs"):
        pick = (rand(n) ** 2 * 8).long().clamp_(max=7)
        s["tokens"] = ids.gather(1, pick[:, None])[:, 0].contiguous()
        if case["op"] == "logprobs_train":        # advantages, and an entropy bonus
            s["g_logp"] = torch.randn(n, generator=g, device="cuda") / n
            s["g_entropy"] = -0.01 * (1 + rand(n)) / n
        return s
    s["ids"] = ids[:, :k].to(torch.int32).contiguous()
    s["teacher"] = (torch.linspace(9.0, 0.0, k, device="cuda") + 1.5 * rand(n, k)).contiguous()
    if case["short"]:                             # answers that list fewer ids end in -1
        s["ids"][n // 2:, (k + 1) // 2:] = -1
    # what the teacher's other tokens weigh: 2 to 25 % of it
    s["lse"] = (torch.logsumexp(s["teacher"] / case["temperature"], 1) + 0.02 + 0.25 * rand(n)) if case["tail"] else None
    w = (0.5 + rand(n)) / n
    if case["masked_rows"]:
        w[n - case["masked_rows"]:] = 0.0
    s["weight"] = w
    return s


# --- the plain form: 32-bit elementary operations --------------------------------------------------------------------

def _softmax(x, temperature):
    """s - m, its exponentials and their sum."""
    d = x.float() / temperature
    d = d - d.amax(1, keepdim=True)
    e = d.exp()
    return d, e, e.sum(1, keepdim=True)


def _top(x, k):
    """Ids of the k largest, ties by the lowest id: 64-bit keys of value and id, no two alike."""
    bits = (x.float() + 0.0).contiguous().view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    key = order * 2 ** 32 + (2 ** 32 - 1 - torch.arange(x.shape[1], device=x.device))
    return (2 ** 32 - 1 - (key.topk(k, dim=1).values & (2 ** 32 - 1)))


def _plain_logprobs(s):
    case, t = s["case"], s["tokens"][:, None]
    d, e, z = _softmax(s["x"], case["temperature"])
    logz = z.log()
    p = e / z
    plogp = torch.where(p > 0, p * (d - logz), 0.0)
    h = -plogp.sum(1, keepdim=True)
    out = {"logp": (d.gather(1, t) - logz)[:, 0], "entropy": h[:, 0]}
    if case["op"] == "logprobs_train":
        a, b = s["g_logp"][:, None], s["g_entropy"][:, None]
        grad = -a * p - b * (plogp + p * h)
        grad.scatter_add_(1, t, a)
        out["grad"] = (grad / case["temperature"]).to(s["x"].dtype)
    elif case["k"]:
        top = _top(s["x"], case["k"])
        out["top_ids"], out["top_logp"] = top.int(), d.gather(1, top) - logz
    return out


def _plain_distill(s):
    case = s["case"]
    d, e, z = _softmax(s["x"], case["temperature"])
    valid = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    y = torch.where(valid, s["teacher"] / case["temperature"], -math.inf)
    if case["tail"]:
        logq = y - s["lse"][:, None]
        q = logq.exp()
    else:
        y = y - y.amax(1, keepdim=True)
        q = y.exp()
        total = q.sum(1, keepdim=True)
        logq, q = y - total.log(), q / total
    logp = d.gather(1, ids) - z.log()
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    if case["tail"]:
        rest = e.scatter_add(1, ids, torch.where(valid, -e.gather(1, ids), 0.0)).sum(1, keepdim=True)
        r = (1 - q.sum(1, keepdim=True)).clamp(min=0)
        loss = loss + torch.where(r > 0, r * (r.log() - rest.log() + z.log()), 0.0)[:, 0]
    if case["op"] == "distill":
        return {"loss": loss}
    w = s["weight"][:, None]
    p = e / z
    grad = p * q.sum(1, keepdim=True)
    if case["tail"]:
        # a token that is not listed has its share of the rest: p - r p / p_rest
        inside = torch.zeros_like(p).scatter_add_(1, ids, valid.float())
        grad = p * (q.sum(1, keepdim=True) + r) - torch.where(inside > 0, 0.0, p * (r * z / rest))
    grad = (grad.scatter_add_(1, ids, -q) * (w / case["temperature"])).to(s["x"].dtype)
    return {"loss": loss * s["weight"] if case["op"] == "distill_fused" else loss, "grad": grad}


# --- the framework's operators ----------------------------------------------------------------------------------------

def _own(s):
    from quantized_optimizer_state_gb300 import losses
    case, x = s["case"], s["x"]
    if case["op"] == "logprobs":
        o = losses.token_logprobs(x, s["tokens"], top_k=case["k"], temperature=case["temperature"])
        out = {"logp": o.logp, "entropy": o.entropy}
        if case["k"]:
            out["top_ids"], out["top_logp"] = o.top_ids, o.top_logp
        return out
    if case["op"] == "logprobs_train":
        x = x.detach().requires_grad_(True)
        o = losses.token_logprobs(x, s["tokens"], temperature=case["temperature"])
        grad, = torch.autograd.grad((o.logp, o.entropy), x, (s["g_logp"], s["g_entropy"]))
        return {"logp": o.logp.detach(), "entropy": o.entropy.detach(), "grad": grad}
    how = dict(temperature=case["temperature"], teacher_temperature=case["temperature"], tail=case["tail"],
               teacher_lse=s["lse"])
    if case["op"] == "distill":
        return {"loss": losses.distill_loss(x, s["ids"], s["teacher"], **how)}
    if case["op"] == "distill_train":
        x = x.detach().requires_grad_(True)
        loss = losses.distill_loss(x, s["ids"], s["teacher"], **how)
        grad, = torch.autograd.grad(loss, x, s["weight"])
        return {"loss": loss.detach(), "grad": grad}
    loss, grad = losses.distill_loss_grad(x, s["ids"], s["teacher"], row_weight=s["weight"], **how)
    return {"loss": loss, "grad": grad}


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return (_plain_logprobs if state["case"]["op"].startswith("logprobs") else _plain_distill)(state)


def work(case):
    n, v, k, b = case["rows"], case["vocab"], case["k"], BYTES[case["dtype"]]
    read = (n - case["masked_rows"]) * v * b
    grad = n * v * b if case["op"] in ("logprobs_train", "distill_train", "distill_fused") else 0
    small = n * (16 + 8 * k + 4 * bool(case["tail"]))
    # by element: the difference from the maximum, its exponential, the sum, the weighted sum; for a gradient twice that
    return {"bytes": read + grad + small, "flops": n * v * (12 if grad else 6)}


# --- 64 bits, from the definitions ------------------------------------------------------------------------------------

def _exact_rows(s, a, b):
    case = s["case"]
    x = s["x"][a:b].double() / case["temperature"]
    n, v = x.shape
    at = torch.arange(n, device=x.device)
    logp = x - torch.logsumexp(x, 1, keepdim=True)
    if case["op"].startswith("logprobs"):
        p = logp.exp()
        h = -torch.nansum(p * logp, 1)
        out = {"logp": logp[at, s["tokens"][a:b]], "entropy": h}
        if case["op"] == "logprobs_train":
            ga, gb = s["g_logp"][a:b].double(), s["g_entropy"][a:b].double()
            grad = -p * ga[:, None] - gb[:, None] * torch.nan_to_num(p * (logp + h[:, None]), nan=0.0)
            grad[at, s["tokens"][a:b]] += ga
            out["grad"] = grad / case["temperature"]
        elif case["k"]:
            out["top_ids"], out["top_logp"] = None, logp.sort(1, descending=True).values[:, :case["k"]].clone()
        return out
    ids, y = s["ids"][a:b].long(), s["teacher"][a:b].double() / case["temperature"]
    there = ids >= 0
    # the teacher as a whole distribution over the vocabulary and, with a tail, one outcome more
    y = y - (s["lse"][a:b].double()[:, None] if case["tail"] else
             torch.logsumexp(y.masked_fill(~there, -math.inf), 1, keepdim=True))
    full = torch.zeros((n, v + 1), dtype=torch.float64, device=x.device)
    full.scatter_(1, torch.where(there, ids, v), torch.where(there, y.exp(), 0.0))
    full[:, v] = 0.0
    q, listed_ = full[:, :v], full[:, :v] > 0
    p = logp.exp()
    loss = torch.nansum(torch.where(listed_, q * (q.log() - logp), 0.0), 1)
    grad = p - q
    if case["tail"]:
        r = 1 - q.sum(1)
        rest = p.masked_fill(listed_, 0.0).sum(1)
        loss = loss + r * (r / rest).log()
        grad = grad - (p * (r / rest)[:, None]).masked_fill(listed_, 0.0)
    w = s["weight"][a:b].double()
    out = {"loss": loss * w if case["op"] == "distill_fused" else loss}
    if case["op"] != "distill":
        out["grad"] = grad * (w / case["temperature"])[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    rows = max(1, 2 ** 27 // case["vocab"])       # 1 GB a block in 64 bits
    with torch.no_grad():
        parts = [_exact_rows(s, a, min(a + rows, case["rows"])) for a in range(0, case["rows"], rows)]
        return {key: None if parts[0][key] is None else torch.cat([q[key] for q in parts]) for key in parts[0]}
