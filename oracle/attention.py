"""Attention with capped, biased and masked scores in 64 bits (numpy), head by
head from the definition, and the forward-error bounds its bf16 form may have.

    z = scale q.k,  c = cap tanh(z / cap),  s = c - slope |p_i - j|,
    P = softmax over the visible keys (zero where none is), o = P v

No code here is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8        # half an ulp of bf16, relative
# Everything the bf16 form computes in fp32 (scores over at most 128 products,
# the exponential, sums): a relative error of P below 2^-11 for the scores the
# tests draw (sum |q k| scale <= 64: 64 * 128 * 2^-24 = 2^-11).
F = 2.0 ** -11


def visible(q_len, k_len, causal=False, prefix=0, q_docs=None, k_docs=None):
    i = np.arange(q_len)[:, None] + (k_len - q_len)
    j = np.arange(k_len)[None]
    m = np.ones((q_len, k_len), bool)
    if causal:
        m = (j <= i) | (j < prefix)
    if q_docs is not None:
        m = m & (q_docs[:, None] == k_docs[None]) & (q_docs[:, None] >= 0)
    return m


def head(q, k, v, *, scale, see, cap=0.0, slope=0.0):
    """P, dc/dz, o and lse of one head (q [q_len, d], k and v [k_len, d])."""
    q_len, k_len = see.shape
    # what padding holds is never used
    q = np.where(see.any(1)[:, None], q, 0.0)
    k = np.where(see.any(0)[:, None], k, 0.0)
    v = np.where(see.any(0)[:, None], v, 0.0)
    z = scale * (q @ k.T)
    slope_z = np.ones_like(z)
    if cap:
        t = np.tanh(z / cap)
        z, slope_z = cap * t, 1.0 - t * t
    far = np.abs(np.arange(q_len)[:, None] + (k_len - q_len) - np.arange(k_len)[None])
    s = np.where(see, z - slope * far, -np.inf)
    top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
    top = np.where(np.isinf(top), 0.0, top)
    e = np.exp(s - top)
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.log(total[:, 0]) + top[:, 0]
    p = e / np.where(total == 0, 1.0, total)
    return p, slope_z, p @ v, lse, (q, k, v)


def head_backward(do, p, slope_z, o, qkv, *, scale, see):
    q, k, v = qkv
    do = np.where(see.any(1)[:, None], do, 0.0)
    dv = p.T @ do
    dp = do @ v.T
    delta = (do * o).sum(1, keepdims=True)
    dz = p * (dp - delta) * slope_z
    return scale * dz @ k, scale * dz.T @ q, dv, dz, do


def run(q, k, v, do=None, *, scale, causal=False, cap=0.0, slopes=None, prefix=None,
        q_docs=None, k_docs=None):
    """All heads (float64 [batch, len, heads, dim]).  Returns a dict of the
    outputs and, under "bound", how far the bf16 form may be from each."""
    B, sq, hq, d = q.shape
    sk, hk = k.shape[1:3]
    grp = hq // hk
    out = {"o": np.zeros_like(q), "lse": np.zeros((B, hq, sq))}
    bound = {"o": np.zeros_like(q)}
    if do is not None:
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            out[n], bound[n] = np.zeros_like(t), np.zeros_like(t)
    for b in range(B):
        see = visible(sq, sk, causal, 0 if prefix is None else prefix[b],
                      None if q_docs is None else q_docs[b], None if k_docs is None else k_docs[b])
        for h in range(hq):
            g = h // grp
            p, sl, o, lse, qkv = head(q[b, :, h], k[b, :, g], v[b, :, g], scale=scale, see=see,
                                      cap=cap, slope=0.0 if slopes is None else slopes[h])
            out["o"][b, :, h], out["lse"][b, h] = o, lse
            qq, kk, vv = qkv
            pv = p @ np.abs(vv)
            # P rounded to bf16, the output rounded to bf16, fp32 in between
            bound["o"][b, :, h] = (2 * U + F) * pv
            if do is None:
                continue
            dq, dk, dv, dz, e = head_backward(do[b, :, h], p, sl, o, qkv, scale=scale, see=see)
            out["dq"][b, :, h] = dq
            out["dk"][b, :, g] += dk
            out["dv"][b, :, g] += dv
            bound["dv"][b, :, g] += (2 * U + F) * (p.T @ np.abs(e))
            # dz: rounded to bf16, from P, dP and delta in fp32, delta from an
            # output that is off by its own bound
            off = p * sl * ((np.abs(e) * (2 * U + F) * pv).sum(1, keepdims=True)
                            + F * (np.abs(e) @ np.abs(vv).T + (np.abs(e) * pv).sum(1, keepdims=True)))
            dzb = (2 * U + 2 * F) * np.abs(dz) + off
            bound["dq"][b, :, h] = scale * dzb @ np.abs(kk)
            bound["dk"][b, :, g] += scale * dzb.T @ np.abs(qq)
    out["bound"] = bound
    return out
