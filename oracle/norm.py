"""fp64 definitions of the dropout mask and of the root-mean-square norm with the
residual's addition (numpy; nothing shared with the GPU path).

The generator is Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011); the norm is that of ch05
"Acceleration principles: Triton kernels and fused LoRA", §5.4.
"""
from __future__ import annotations

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
LOW = np.uint64(0xFFFFFFFF)


def philox(counter, key, rounds=10):
    """Four words of 32 bits from a counter of four and a key of two (Python integers)."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p, q = M0 * c[0], M1 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return c


def words(rows, cols, seed, offset, first_row=0):
    """[rows, cols] words: word(n, c) of row first_row + n."""
    blocks = (cols + 3) // 4
    n = np.arange(first_row, first_row + rows, dtype=np.uint64)[:, None]
    b = np.arange(blocks, dtype=np.uint64)[None]
    c = [b + 0 * n, (n & LOW) + 0 * b, (n >> np.uint64(32)) + 0 * b,
         np.full((rows, blocks), offset, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = np.uint64(M0) * c[0], np.uint64(M1) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & LOW,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & LOW]
        k = [(k[0] + W0) & 0xFFFFFFFF, (k[1] + W1) & 0xFFFFFFFF]
    return np.stack(c, -1).reshape(rows, 4 * blocks)[:, :cols]


def dropout(x, p, seed, offset, first_row=0):
    """x [rows, cols] fp64."""
    t = int(round(p * 2 ** 32))
    keep = words(*x.shape, seed, offset, first_row) >= t
    return np.where(keep, x * (2.0 ** 32 / (2 ** 32 - t)), 0.0)


def forward(h, w, eps):
    """(y, rstd) of the rows of h."""
    r = 1.0 / np.sqrt(np.mean(h * h, -1) + eps)
    return h * r[:, None] * w, r


def backward(dy, h, w, r, dh=None):
    """(gradient of h, dw)."""
    hat = h * r[:, None]
    g = dy * w
    d = r[:, None] * (g - hat * np.mean(g * hat, -1, keepdims=True))
    return (d if dh is None else d + dh), np.sum(dy * hat, 0)


def row_scale(y):
    """2^e of each row, e the smallest integer >= -126 with max|y| <= 448 2^e."""
    top = np.max(np.abs(y), -1)
    e = np.where(top > 0, np.ceil(np.log2(np.where(top > 0, top, 1.0) / 448.0)), 0)
    return 2.0 ** np.maximum(e, -126)
