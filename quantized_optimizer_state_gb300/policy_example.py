"""Policy training of a small language model with what a step holds in memory in 8
bits, the operators together as a training loop uses them:

* blocks of :func:`.activations.rms_norm`, :func:`.activations.linear` and a gated
  :func:`.activations.activation`, whose inputs are kept as codes for the backward pass;
* the policy samples a token for each context, which a rule rewards;
  :func:`.losses.token_logprobs` writes down what it, and a frozen reference, made of them;
* :func:`.losses.policy_loss_grad` gives the clipped loss and the gradient of the
  logits in one call, over a few steps on the same tokens;
* :class:`.optim.FlashAdamW` steps its compressed state.

The model predicts a token from one before it. The data is synthetic and the
weights random.

    python -m quantized_optimizer_state_gb300.policy_example [--vocab 2003] [--steps 20]
"""
from __future__ import annotations

import argparse
import copy

import torch

from . import activations as act
from .losses import policy_loss_grad, token_logprobs
from .optim import FlashAdamW


class Block(torch.nn.Module):
    """h + down(swiglu(gate_up(norm(h))))"""

    def __init__(self, dim: int, hidden: int, device):
        super().__init__()
        self.norm = torch.nn.Parameter(torch.ones(dim, device=device))
        self.gate_up = torch.nn.Parameter(torch.randn(2 * hidden, dim, device=device) / dim ** 0.5)
        self.down = torch.nn.Parameter(torch.randn(dim, hidden, device=device) / hidden ** 0.5)

    def forward(self, h: torch.Tensor) -> torch.Tensor:
        x = act.rms_norm(h, self.norm)
        return h + act.linear(act.activation(act.linear(x, self.gate_up), "swiglu"), self.down)


class Policy(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, hidden: int, blocks: int, device):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, dim, device=device)
        self.blocks = torch.nn.ModuleList([Block(dim, hidden, device) for _ in range(blocks)])
        self.norm = torch.nn.Parameter(torch.ones(dim, device=device))
        self.head = torch.nn.Parameter(torch.randn(vocab, dim, device=device) / dim ** 0.5)

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        h = self.embed(tokens)
        for block in self.blocks:
            h = block(h)
        return act.linear(act.rms_norm(h, self.norm), self.head)


def run(vocab: int = 2003, dim: int = 128, hidden: int = 344, blocks: int = 2, contexts: int = 64, samples: int = 16,
        epochs: int = 2, kl_weight: float = 0.02, steps: int = 20, lr: float = 3e-3, seed: int = 0, log=None):
    """Trains the policy to answer every context with a token of its own half of the
    vocabulary; gives the mean rewards and losses by step."""
    device = torch.device("cuda")
    torch.manual_seed(seed)
    policy = Policy(vocab, dim, hidden, blocks, device)
    opt = FlashAdamW(policy.parameters(), lr=lr, weight_decay=0.0)      # FP32 weights become BF16 + correction
    reference = copy.deepcopy(policy).requires_grad_(False)
    seen = torch.randint(0, vocab, (contexts,), device=device)
    rewards, losses = [], []
    for step in range(steps):
        with torch.no_grad():
            logits = policy(seen)
            tokens = torch.multinomial(torch.softmax(logits.float(), 1), samples, replacement=True)    # [contexts, samples]
        reward = ((tokens < vocab // 2) == (seen[:, None] < vocab // 2)).float()
        advantage = (reward - reward.mean(1, keepdim=True)) / (reward.std(1, keepdim=True) + 1e-3)
        batch = seen.repeat_interleave(samples)
        tokens, advantage = tokens.flatten(), advantage.flatten()
        tokens[::61] = -1                                               # positions that a real batch pads
        weight = torch.where(tokens >= 0, 1.0 / (tokens >= 0).sum(), 0.0)
        with torch.no_grad():
            old = token_logprobs(policy(batch), tokens, entropy=False).logp
            ref = token_logprobs(reference(batch), tokens, entropy=False).logp
        for _ in range(epochs):
            logits = policy(batch)
            o = policy_loss_grad(logits.detach(), tokens, old, advantage, ref_logp=ref, kl_weight=kl_weight,
                                 clip_high=0.28, row_weight=weight)
            logits.backward(o.grad)
            opt.step()
            opt.zero_grad()
        rewards.append(reward.mean())
        losses.append(o.loss.sum())
        if log:
            log(f"step {step:4d}  reward {float(rewards[-1]):.3f}  loss {float(losses[-1]):+.4f}")
    return {"rewards": [float(r) for r in rewards], "losses": [float(l) for l in losses], "policy": policy}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=2003)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--samples", type=int, default=16)
    ap.add_argument("--kl-weight", type=float, default=0.02)
    a = ap.parse_args()
    r = run(vocab=a.vocab, steps=a.steps, samples=a.samples, kl_weight=a.kl_weight, log=print)
    print(f"mean reward {r['rewards'][0]:.3f} -> {r['rewards'][-1]:.3f}")


if __name__ == "__main__":
    main()
