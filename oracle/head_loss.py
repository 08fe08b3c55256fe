"""Softmax cross entropy of a head in 64 bits (numpy), from the definition, with the
gradient of the hidden states and the bounds its bf16 form may have.

    z = c(X W^T), loss_n = logsumexp(z_n) - z_n,t, loss = sum_n g_n loss_n
    dX_n = g_n sum_v (p_nv - [v = t_n]) c'(z) W_v

(ch05 "Acceleration principles: Triton kernels and fused LoRA", §5.7.)  No code
here is shared with the CUDA path.

Bounds.  F = 2^-23: a step of fp32, what an accumulation may cut off.
  z: dim products, exact in fp32, one after the other: dim F sum |x w|, and what
     the cap's formula may be off by: 8 F |z|.  dz is the largest of a row.
  losses: two such errors (the sums of exponentials and the target), and the
     logarithm's and the sums' own: 40 F of 1 + |loss|.
  q = p - [v = t], each rounded to half a step of bf16 (U = 2^-8), off by 3 dz
     through the exponentials, the sum and the target, and 40 F:
     dX: (U + 3 dz + 40 F + vocab F) sum |q W| for the products, whose terms are
     added one after the other, and one rounding U |dX|.
"""
from __future__ import annotations

import numpy as np

F = 2.0 ** -23
U = 2.0 ** -8


def run(x, w, targets, weights=None, cap=0.0, mean=True, gradient=True):
    """x [rows, dim], w [vocab, dim] fp64; targets [rows].  A dict of loss, losses, dx
    and their bounds e_loss, e_losses, e_dx."""
    live = targets >= 0
    g = live * (1.0 if weights is None else np.where(live, weights, 0.0))
    total = g.sum()
    if mean and total != 0:
        g = g / total
    raw = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    z, slope = raw, np.ones_like(raw)
    if cap:
        z = cap * np.tanh(raw / cap)
        a = np.exp(-2 * np.abs(raw) / cap)
        slope = 4 * a / (1 + a) ** 2
    dz = np.max(x.shape[1] * F * size + 8 * F * np.abs(z), -1)
    at = np.arange(len(x)), np.where(live, targets, 0)
    rest = z - z[at][:, None]
    rest[at] = -np.inf
    top = np.maximum(np.max(rest, -1), 0)
    s = np.sum(np.exp(rest - top[:, None]), -1)  # without the target, times exp(-top)
    losses = np.where(top > 0, top + np.log(s + np.exp(-top)), np.log1p(s))
    losses = np.where(live, losses, 0.0)
    e_losses = live * (2 * dz + 40 * F * (1 + np.abs(losses)))
    out = dict(loss=float(np.sum(g * losses)), losses=losses, e_losses=e_losses,
               e_loss=float(np.sum(np.abs(g) * (e_losses + F * np.abs(losses)))) + 1e-37)
    if not gradient:
        return out
    q = np.exp(rest - top[:, None]) / (s + np.exp(-top))[:, None]
    q[at] = -s / (s + np.exp(-top))
    q = q * slope
    dx = g[:, None] * (q @ w)
    each = np.abs(g)[:, None] * (np.abs(q) @ np.abs(w))
    out["dx"] = dx
    out["e_dx"] = (U + 3 * dz + 40 * F + w.shape[0] * F)[:, None] * each * 1.01 + U * np.abs(dx) + 1e-37
    return out
