"""Distillation of a small language model into a smaller one, with the loss
operators and the fused optimizer together:

* a teacher scores a batch of tokens; :func:`.losses.token_logprobs` writes down
  its top alternatives and their log probabilities;
* the student's logits go through :func:`.losses.distill_loss_grad`, which gives
  the loss and the gradient of the logits in one call (padding has weight 0);
* the gradient runs back through the student and
  :class:`.optim.FlashAdamW` steps its compressed state.

Both models predict a token from the one before it (an embedding, a
non-linearity, a head): enough to have real logits over a whole vocabulary. The
data is synthetic and the weights random.

    python -m quantized_optimizer_state_gb300.distill_example [--vocab 50257] [--steps 100]
"""
from __future__ import annotations

import argparse

import torch

from .losses import distill_loss_grad, token_logprobs
from .optim import FlashAdamW


class NextToken(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, device, scale: float):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, dim, device=device)
        self.head = torch.nn.Linear(dim, vocab, bias=False, device=device)
        torch.nn.init.normal_(self.embed.weight)
        torch.nn.init.normal_(self.head.weight, std=scale / dim ** 0.5)

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        h = torch.tanh(self.embed(tokens))
        return h.to(self.head.weight.dtype) @ self.head.weight.t()


def run(vocab: int = 50257, teacher_dim: int = 128, student_dim: int = 64, batch: int = 1024, contexts: int = 64,
        top_k: int = 32, temperature: float = 2.0, steps: int = 100, lr: float = 1e-2, seed: int = 0, log=None):
    """Trains the student; gives the mean KL of the first and of the last step and the
    student's mean log probability of the teacher's best token before and after."""
    device = torch.device("cuda")
    torch.manual_seed(seed)
    teacher = NextToken(vocab, teacher_dim, device, 8.0).to(torch.bfloat16).requires_grad_(False)
    student = NextToken(vocab, student_dim, device, 1.0)
    opt = FlashAdamW(student.parameters(), lr=lr, weight_decay=0.0)     # FP32 weights become BF16 + correction
    seen = torch.randint(0, vocab, (contexts,), device=device)          # the contexts that the data holds
    weight = torch.full((batch,), 1.0 / (batch - batch // 16), device=device)
    weight[batch - batch // 16:] = 0.0                                  # padding at the end of the batch

    def best_token():
        best = token_logprobs(teacher(seen), top_k=1, entropy=False).top_ids[:, 0].long()
        with torch.no_grad():
            return token_logprobs(student(seen), best).logp.mean()

    before, kl = best_token(), []
    for step in range(steps):
        tokens = seen[torch.randint(0, contexts, (batch,), device=device)]
        told = token_logprobs(teacher(tokens), top_k=top_k, temperature=temperature, entropy=False)
        logits = student(tokens)
        loss, grad = distill_loss_grad(logits.detach(), told.top_ids, told.top_logp, row_weight=weight,
                                       temperature=temperature, tail=True)
        logits.backward(grad)
        opt.step()
        opt.zero_grad()
        kl.append(loss.sum())
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  KL {float(kl[-1]):.4f}")
    return {"kl_first": float(kl[0]), "kl_last": float(kl[-1]), "logp_before": float(before),
            "logp_after": float(best_token())}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=50257)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--batch", type=int, default=1024)
    ap.add_argument("--top-k", type=int, default=32)
    ap.add_argument("--temperature", type=float, default=2.0)
    a = ap.parse_args()
    r = run(vocab=a.vocab, batch=a.batch, top_k=a.top_k, temperature=a.temperature, steps=a.steps, log=print)
    print(f"KL {r['kl_first']:.4f} -> {r['kl_last']:.4f}; log probability of the teacher's best token "
          f"{r['logp_before']:.3f} -> {r['logp_after']:.3f}")


if __name__ == "__main__":
    main()
