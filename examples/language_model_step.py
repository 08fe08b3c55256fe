"""Fine-tuning steps of a small language model's MLP blocks and head, end to end.

Token embeddings go through blocks of norm -> fp8 LoRA layer up -> LoRA layer
down, each branch dropped out before it joins the residual stream; the last norm
feeds the frozen head's cross entropy, whose gradient comes back through all of
them into the adapters and the norms' weights.  Prompt tokens do not count.  Then
the tuned model scores a continuation.

    python examples/language_model_step.py [--steps 5] [--tokens 512]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rank_linear_gb300 as rl  # noqa: E402


class Model:
    """h += dropout(down(dropout(up(norm(h))))) per block; logits = norm(h) head^T."""

    def __init__(self, vocab=5003, width=256, inner=512, blocks=2, rank=8, alpha=16.0, p=0.1, softcap=0.0,
                 seed=0, device="cuda:0"):
        self.alpha, self.p, self.softcap = alpha, p, softcap
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=device)
        self.embed = r(vocab, width).bfloat16()
        self.head = (r(vocab, width) * width ** -0.5).bfloat16()
        self.norms = [torch.ones(width, device=device).requires_grad_() for _ in range(blocks + 1)]
        self.up_w = [(r(inner, width) * width ** -0.5).bfloat16() for _ in range(blocks)]
        self.up_q = [rl.quantize_w_fp8(w) for w in self.up_w]
        self.down_w = [(r(width, inner) * inner ** -0.5).bfloat16() for _ in range(blocks)]
        self.adapters = []
        for _ in range(blocks):
            pair = [(r(rank, width) * width ** -0.5).bfloat16(), (r(inner, rank) * 0.05).bfloat16(),
                    (r(rank, inner) * inner ** -0.5).bfloat16(), (r(width, rank) * 0.05).bfloat16()]
            self.adapters.append([t.requires_grad_() for t in pair])

    def parameters(self):
        return self.norms + [t for a in self.adapters for t in a]

    def hidden(self, tokens, seed, train=True):
        """The last norm's output [..., width]."""
        stream, branch = self.embed[tokens], None
        for i, (a_up, b_up, a_down, b_down) in enumerate(self.adapters):
            # the branch of the block before joins the stream inside the norm
            x, rest = (stream, {}) if branch is None else \
                (branch, dict(residual=stream, dropout=self.p if train else 0.0, seed=seed, offset=i))
            out = rl.rms_norm(x, self.norms[i], eps=1e-5, fp8=True, **rest)
            y, codes, scale = out[0], out[-2], out[-1]
            stream = out[1] if rest else stream
            u = rl.lora_linear_fp8(y, self.up_q[i], a_up, b_up, self.alpha, rows=(codes, scale))
            if train:
                u = rl.dropout(u, self.p, seed, 100 + i)
            branch = rl.lora_linear(u, self.down_w[i], a_down, b_down, self.alpha)
        y, _ = rl.rms_norm(branch, self.norms[-1], residual=stream, eps=1e-5,
                           dropout=self.p if train else 0.0, seed=seed, offset=len(self.adapters))
        return y

    def loss(self, tokens, targets, seed, train=True):
        return rl.cross_entropy(self.hidden(tokens, seed, train), self.head, targets, softcap=self.softcap)


def main(steps=5, tokens=512, device="cuda:0"):
    model = Model(device=device)
    g = torch.Generator(device=device).manual_seed(1)
    vocab = model.embed.shape[0]
    ids = torch.randint(0, vocab, (2, tokens), generator=g, device=device)
    targets = torch.roll(ids, -1, 1)
    targets[:, :tokens // 3] = -100   # the prompt
    targets[:, -1] = -100             # nothing follows
    params = model.parameters()
    for t in params:
        t.grad = torch.zeros_like(t)
    clip = rl.GradClip(params=params)
    losses = []
    for step in range(steps):
        for t in params:
            t.grad.zero_()
        loss, _ = model.loss(ids, targets, seed=step)
        loss.backward()
        norm = clip.clip(1.0)
        with torch.no_grad():
            for t in params:
                t -= 0.5 * t.grad
        losses.append(loss.item())
        print(f"step {step}: loss {losses[-1]:.4f}, gradient norm {norm.item():.4f}")
    with torch.no_grad():
        _, each = model.loss(ids[:1], targets[:1], seed=0, train=False)
    count = int((targets[0] >= 0).sum())
    score = -each.sum().item() / count
    print(f"mean log-probability of the first sequence's continuation: {score:.4f}")
    rl.device_status()
    return losses, score


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    main(a.steps, a.tokens)
