"""Fine-tuning steps of one attention block, and its serving form, end to end.

Packed documents go through the q, k and v LoRA layers, rotary positions, the
masked attention and the o LoRA layer; the loss's gradients come back through
all of them into the eight adapter matrices, are clipped by their global norm
and applied.  Then a prompt's k and v are kept as a cache and new tokens are
attended one at a time.

    python examples/attention_block_step.py [--steps 5] [--tokens 1024]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rank_linear_gb300 as rl  # noqa: E402

NAMES = ("q", "k", "v", "o")


class AttentionBlock:
    """y = o(attention(rotary(q(x)), rotary(k(x)), v(x))), every product a LoRA
    layer over a frozen bf16 weight."""

    def __init__(self, width=1024, heads=8, kv_heads=2, rank=16, alpha=32.0, softcap=0.0, seed=0,
                 device="cuda:0"):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, width // heads
        self.alpha, self.softcap = alpha, softcap
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=device)
        outs = dict(q=width, k=kv_heads * self.dim, v=kv_heads * self.dim, o=width)
        self.W = {n: (r(outs[n], width) * width ** -0.5).bfloat16() for n in NAMES}
        self.A = {n: (r(rank, width) * width ** -0.5).bfloat16() for n in NAMES}
        self.B = {n: (r(outs[n], rank) * 0.1).bfloat16() for n in NAMES}
        self.adapters = [t for n in NAMES for t in (self.A[n], self.B[n])]
        for t in self.adapters:
            t.requires_grad_()
            t.grad = torch.zeros_like(t)  # stays where it is: the clip's plan holds its address
        self.freqs = rl.rotary_frequencies(self.dim, base=10000.0, device=device)

    def project(self, name, x):
        return rl.lora_linear(x, self.W[name], self.A[name], self.B[name], self.alpha)

    def qkv(self, x, positions):
        b, s, _ = x.shape
        q = self.project("q", x).view(b, s, self.heads, self.dim)
        k = self.project("k", x).view(b, s, self.kv_heads, self.dim)
        v = self.project("v", x).view(b, s, self.kv_heads, self.dim)
        q, k = rl.rotary(q, k, positions, self.freqs)
        return q, k, v

    def forward(self, x, positions, documents):
        q, k, v = self.qkv(x, positions)
        o = rl.attention(q, k, v, causal=True, softcap=self.softcap, documents=documents)
        return self.project("o", o.flatten(2))

    def step_token(self, x, length, k_cache, v_cache):
        """One new token per sequence: x [batch, width]; length int32 [batch] tokens
        are already in the caches, which take the new one."""
        b = x.shape[0]
        q, k, v = self.qkv(x[:, None], length[:, None].long())
        at = torch.arange(b, device=x.device)
        k_cache[at, length.long()] = k[:, 0]
        v_cache[at, length.long()] = v[:, 0]
        o = rl.attention_decode(q[:, 0], k_cache, v_cache, length + 1, softcap=self.softcap)
        return self.project("o", o.flatten(1))


def packed(lengths, pad, device):
    """(documents, positions within each) of one packed row; -1 for the padding."""
    docs = sum(([i] * n for i, n in enumerate(lengths)), []) + [-1] * pad
    pos = sum((list(range(n)) for n in lengths), []) + [0] * pad
    return (torch.tensor([docs], dtype=torch.int32, device=device),
            torch.tensor([pos], device=device))


def main(steps=5, tokens=1024, device="cuda:0"):
    block = AttentionBlock(device=device)
    width = block.W["q"].shape[1]
    g = torch.Generator(device=device).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=device).bfloat16()
    lengths = [tokens // 2, tokens // 3, tokens // 8]
    documents, positions = packed(lengths, tokens - sum(lengths), device)
    x, target = r(1, tokens, width), r(1, tokens, width)
    live = (documents >= 0)[..., None].float()

    clip = rl.GradClip(params=block.adapters)
    losses = []
    for step in range(steps):
        y = block.forward(x, positions, documents)
        loss = ((y.float() - target.float()).square() * live).mean()
        for t in block.adapters:
            t.grad.zero_()
        loss.backward()
        norm = clip.clip(0.05)
        with torch.no_grad():
            for t in block.adapters:
                t -= 4.0 * t.grad
        losses.append(loss.item())
        print(f"step {step}: loss {losses[-1]:.5f}, gradient norm {norm.item():.4f}")

    # serving: the first document as a prompt, its last token again as a new one
    n = lengths[0]
    with torch.no_grad():
        prompt = x[:, :n]
        q, k, v = block.qkv(prompt, positions[:, :n])
        whole = block.forward(prompt, positions[:, :n], None)[:, -1]
        k_cache = torch.zeros(1, n + 16, block.kv_heads, block.dim, dtype=x.dtype, device=device)
        v_cache = torch.zeros_like(k_cache)
        k_cache[:, :n - 1], v_cache[:, :n - 1] = k[:, :-1], v[:, :-1]
        length = torch.tensor([n - 1], dtype=torch.int32, device=device)
        token = block.step_token(prompt[:, -1], length, k_cache, v_cache)
    apart = (token.float() - whole.float()).norm() / whole.float().norm()
    print(f"the prompt's last token against a new token over the cache: {apart.item():.1e} apart")
    rl.device_status()
    return losses, apart.item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    main(a.steps, a.tokens)
