"""Cases of the operators between and after the LoRA layers of a fine-tuning step:
rotary positions, masked attention (training, prompts, one new token), and the
clipping of gradients by their global norm.

Where `own` is false, `run` computes an operator from elementary torch
operations in 32 bits; where it is true, it calls this framework.  `exact`
gives the same outputs from the definitions in 64 bits.

Sizes: a head of 128, 32 query heads and widths 4096 / 14336 are those of the
framework's Llama-3-8B layers, 40 heads and widths 5120 / 27648 those of its
wide FFN workload, ranks 16 and 128 its adapters'; the rest is generic.
"""
import math

import torch

own = False

DEV = "cuda:0"
BF16, FP32 = "bf16", "fp32"
TORCH = {BF16: torch.bfloat16, FP32: torch.float32}
SIZE = {BF16: 2, FP32: 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # serving: one new token of 8 sequences, far out in a context stretched 16 times
        rotary("rotary_one_token", batch=8, seq=1, q_heads=32, k_heads=8, dim=128, rot=128,
               interleaved=False, scaling="ramp", far=120000, dtype=BF16, train=False, fused=True),
        # training: a q_proj / k_proj step of 4096 tokens, forward and backward, q and k views of one q|k|v output
        rotary("rotary_train", batch=1, seq=4096, q_heads=32, k_heads=8, dim=128, rot=128,
               interleaved=False, scaling="none", far=0, dtype=BF16, train=True, fused=True),
        # a long odd prompt, half of each head rotated in neighbouring pairs, kept in fp32
        rotary("rotary_part_fp32", batch=3, seq=5461, q_heads=40, k_heads=8, dim=128, rot=64,
               interleaved=True, scaling="bands", far=60000, dtype=FP32, train=False, fused=False),
        # a short odd batch with a distance bias: latency of one small call
        attention("attn_short_bias", batch=3, q_len=257, k_len=257, q_heads=8, k_heads=2, dim=64,
                  causal=True, docs=0, pad=0, prefix=0, cap=0.0, bias=True, train=False),
        # the middle piece of a long prompt: its last 2048 tokens against all 16000 so far
        attention("attn_prompt_piece", batch=1, q_len=2048, k_len=16000, q_heads=32, k_heads=8,
                  dim=128, causal=True, docs=0, pad=0, prefix=0, cap=0.0, bias=False, train=False),
        # a training step on ragged documents packed into 8192 tokens, the tail padded
        attention("attn_train_packed", batch=1, q_len=8192, k_len=8192, q_heads=32, k_heads=8,
                  dim=128, causal=True, docs=5, pad=75, prefix=0, cap=0.0, bias=False, train=True),
        # a training step with capped scores and a prefix seen by all, odd length
        attention("attn_train_cap_prefix", batch=2, q_len=2047, k_len=2047, q_heads=16, k_heads=4,
                  dim=128, causal=True, docs=0, pad=0, prefix=300, cap=30.0, bias=False, train=True),
        # serving: a ragged batch, one new token each
        decode("token_batch", batch=32, length=8192, ragged=0.9, q_heads=32, k_heads=8, dim=128,
               cap=0.0, bias=False),
        # serving: one sequence with a long cache, capped scores
        decode("token_long", batch=1, length=131071, ragged=0.0, q_heads=32, k_heads=8, dim=128,
               cap=50.0, bias=False),
        # the adapters of one layer's seven products
        clip("clip_one_layer", layers=1, rank=16, width=4096, kv_width=1024, ffn=14336,
             dtypes=BF16, largest=False, clipped=True),
        # the adapters of a 32-layer model
        clip("clip_adapters", layers=32, rank=16, width=4096, kv_width=1024, ffn=14336,
             dtypes=BF16, largest=False, clipped=True),
        # wide adapters of rank 128, gradients accumulated in fp32 beside bf16 ones
        clip("clip_wide_mixed", layers=48, rank=128, width=5120, kv_width=1024, ffn=27648,
             dtypes="mixed", largest=False, clipped=True),
    ]


def rotary(name=None, **kw):
    c = dict(op="rotary", **kw)
    return {"name": name, **c} if name else c


def attention(name=None, **kw):
    c = dict(op="attention", **kw)
    return {"name": name, **c} if name else c


def decode(name=None, **kw):
    c = dict(op="decode", **kw)
    return {"name": name, **c} if name else c


def clip(name=None, **kw):
    c = dict(op="clip", **kw)
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "attention", "attention", "decode", "clip"])
    kh = rng.choice([1, 2, 4, 8])
    qh = kh * rng.choice([1, 2, 4, 5] if kh > 1 else [1, 4, 8])
    if op == "rotary":
        dim = rng.choice([64, 80, 96, 128])
        return rotary(batch=rng.choice([1, 1, 2, 5]), seq=_log_int(rng, 1, 3200), q_heads=qh, k_heads=kh,
                      dim=dim, rot=rng.choice([dim, dim // 2, 32]), interleaved=rng.random() < 0.5,
                      scaling=rng.choice(["none", "linear", "base", "bands", "ramp"]),
                      far=rng.choice([0, 1000, 100000]), dtype=rng.choice([BF16, BF16, FP32]),
                      train=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "decode":
        batch = _log_int(rng, 1, 48)
        return decode(batch=batch, length=_log_int(rng, 1, 200000 // batch), ragged=rng.choice([0.0, 0.5, 1.0]),
                      q_heads=qh, k_heads=kh, dim=rng.choice([64, 80, 96, 128, 128]),
                      cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.3)
    if op == "clip":
        return clip(layers=_log_int(rng, 1, 40), rank=rng.choice([1, 4, 7, 8, 16, 33, 64]),
                    width=rng.choice([1000, 2048, 4096, 5120]), kv_width=rng.choice([250, 1024]),
                    ffn=_log_int(rng, 1501, 14336), dtypes=rng.choice([BF16, FP32, "mixed"]),
                    largest=rng.random() < 0.3, clipped=rng.random() < 0.7)
    train = rng.random() < 0.5
    qh, batch, dim = min(qh, 32), rng.choice([1, 1, 2, 3]), rng.choice([64, 64, 80, 96, 128, 128, 128])
    # at most the listed cases' work where nothing is masked
    k_len = _log_int(rng, 1, int(math.sqrt(4.6e11 / (14 * dim * qh * batch))))
    causal = rng.random() < 0.75
    docs = rng.choice([0, 0, 1, 3, 12]) if k_len >= 64 else 0
    same = train or docs or rng.random() < 0.5
    return attention(batch=batch, q_len=k_len if same else _log_int(rng, 1, k_len), k_len=k_len,
                     q_heads=qh, k_heads=kh, dim=dim, causal=causal,
                     docs=docs, pad=rng.choice([0, k_len // 7]) if docs else 0,
                     prefix=rng.choice([0, 1 + k_len // 5]) if causal else 0,
                     cap=rng.choice([0.0, 0.0, 15.0, 50.0]), bias=rng.random() < 0.3, train=train)


# ------------------------------------------------------------------ work

def _doc_lengths(c):
    """Ragged document lengths of one packed row; the pad tokens belong to none."""
    n = c["k_len"] - c["pad"]
    w = [1.0 + 0.8 * math.sin(1.7 * i + 0.4) for i in range(c["docs"])]
    edges = [int(round(n * sum(w[:i]) / sum(w))) for i in range(c["docs"] + 1)]
    return [b - a for a, b in zip(edges, edges[1:])]


def _visible_pairs(c):
    """Query-key pairs that the mask of one batch entry leaves."""
    q, k = c["q_len"], c["k_len"]
    if not c["docs"]:
        if not c["causal"]:
            return q * k
        p = c["prefix"]
        return sum(max(i + k - q + 1, min(p, k)) for i in range(q))
    total, begin = 0, 0
    for n in _doc_lengths(c):
        if not c["causal"]:
            total += n * n
        else:
            p = min(max(c["prefix"] - begin, 0), n)
            total += n * (n + 1) // 2 + p * (p - 1) // 2
        begin += n
    return total


def _cache_lengths(c):
    b = c["batch"]
    return [max(0, int(round(c["length"] * (1.0 - c["ragged"] * i / max(1, b - 1))))) for i in range(b)]


def _clip_shapes(c):
    """(rows, columns) of the A and B gradients of the seven products of every layer."""
    r, w, kv, f = c["rank"], c["width"], c["kv_width"], c["ffn"]
    one = []
    for d_in, d_out in ((w, w), (w, kv), (w, kv), (w, w), (w, f), (w, f), (f, w)):
        one += [(r, d_in), (d_out, r)]
    return one * c["layers"]


def _clip_dtypes(c):
    n = len(_clip_shapes(c))
    return [(BF16 if i % 2 else FP32) if c["dtypes"] == "mixed" else c["dtypes"] for i in range(n)]


def work(c):
    if c["op"] == "rotary":
        tokens, heads = c["batch"] * c["seq"], c["q_heads"] + c["k_heads"]
        passes = 2 if c["train"] else 1
        return {"bytes": passes * (tokens * heads * c["dim"] * 2 * SIZE[c["dtype"]] + tokens * 8),
                "flops": passes * tokens * heads * c["rot"] * 3}
    if c["op"] == "decode":
        live = sum(_cache_lengths(c))
        return {"bytes": live * c["k_heads"] * c["dim"] * 4 + c["batch"] * c["q_heads"] * c["dim"] * 4 + c["batch"] * 4,
                "flops": live * c["q_heads"] * c["dim"] * 4}
    if c["op"] == "clip":
        size = sum(a * b * SIZE[t] for (a, b), t in zip(_clip_shapes(c), _clip_dtypes(c)))
        count = sum(a * b for a, b in _clip_shapes(c))
        return {"bytes": 2 * size, "flops": 3 * count}
    q = c["batch"] * c["q_len"] * c["q_heads"] * c["dim"] * 2
    k = c["batch"] * c["k_len"] * c["k_heads"] * c["dim"] * 2
    pairs = c["batch"] * c["q_heads"] * _visible_pairs(c)
    if c["train"]:  # q, k, v and do in; o, dq, dk and dv out
        return {"bytes": 4 * q + 4 * k, "flops": 14 * c["dim"] * pairs}
    return {"bytes": 2 * q + 2 * k, "flops": 4 * c["dim"] * pairs}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(TORCH[dtype])


SCALINGS = {
    "none": None,
    # positions divided by 4
    "linear": {"kind": "linear", "factor": 4.0},
    # the base raised so that the slowest pair is stretched 4 times
    "base": {"kind": "base", "factor": 4.0},
    # slow pairs stretched 8 times, fast ones kept, a linear blend of frequencies between
    "bands": {"kind": "bands", "factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0},
    # a ramp over the pair's index between kept and stretched 16 times, with a magnitude
    "ramp": {"kind": "ramp", "factor": 16.0, "original": 8192, "fast": 32.0, "slow": 1.0},
}
ROTARY_BASE = 500000.0


def _angular(c):
    """Radians per position of every rotated pair (64 bits), and the magnitude."""
    r, s = c["rot"], SCALINGS[c["scaling"]]
    base = ROTARY_BASE
    if s and s["kind"] == "base":
        base = base * s["factor"] ** (r / (r - 2)) if r > 2 else base
    w = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if s is None or s["kind"] == "base":
        return w, 1.0
    f = s["factor"]
    if s["kind"] == "linear":
        return [x / f for x in w], 1.0
    if s["kind"] == "bands":
        out = []
        for x in w:
            turns = s["original"] * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - s["low"]) / (s["high"] - s["low"])))
            out.append(keep * x + (1.0 - keep) * x / f)
        return out, 1.0
    at = lambda turns: r * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(s["fast"])), 0), min(math.ceil(at(s["slow"])), r - 1)
    out = []
    for i, x in enumerate(w):
        go = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append((1.0 - go) * x + go * x / f)
    return out, 0.1 * math.log(f) + 1.0


def _rotary_inputs(c, seed):
    g = _generator(seed)
    b, s, hq, hk, d = c["batch"], c["seq"], c["q_heads"], c["k_heads"], c["dim"]

    def pair():
        if c["fused"]:  # one q|k|v output: strided views
            x = _randn(g, (b, s, (hq + 2 * hk), d), c["dtype"])
            return x[:, :, :hq], x[:, :, hq:hq + hk]
        return _randn(g, (b, s, hq, d), c["dtype"]), _randn(g, (b, s, hk, d), c["dtype"])

    q, k = pair()
    dq, dk = pair() if c["train"] else (None, None)
    start = torch.randint(0, c["far"] + 1, (b, 1), generator=g, device=DEV)
    return q, k, dq, dk, start + torch.arange(s, device=DEV)


def _attention_inputs(c, seed):
    g = _generator(seed)
    b, sq, sk, hq, hk, d = (c[n] for n in ("batch", "q_len", "k_len", "q_heads", "k_heads", "dim"))
    # capped scores are only met where some reach the cap
    q = _randn(g, (b, sq, hq, d), BF16, 3.0 if c["cap"] else 1.0)
    k = _randn(g, (b, sk, hk, d), BF16)
    v = _randn(g, (b, sk, hk, d), BF16)
    do = _randn(g, (b, sq, hq, d), BF16) if c["train"] else None
    docs = prefix = None
    if c["docs"]:
        row = sum(([i] * n for i, n in enumerate(_doc_lengths(c))), []) + [-1] * c["pad"]
        docs = torch.tensor([row] * b, dtype=torch.int32, device=DEV)
    if c["prefix"]:
        prefix = torch.full((b,), c["prefix"], dtype=torch.int32, device=DEV)
    return q, k, v, do, docs, prefix, _slopes(c)


def _decode_inputs(c, seed):
    g = _generator(seed)
    b, s, hq, hk, d = (c[n] for n in ("batch", "length", "q_heads", "k_heads", "dim"))
    q = _randn(g, (b, hq, d), BF16, 3.0 if c["cap"] else 1.0)
    k = _randn(g, (b, s, hk, d), BF16)
    v = _randn(g, (b, s, hk, d), BF16)
    lengths = torch.tensor(_cache_lengths(c), dtype=torch.int32, device=DEV)
    return q, k, v, lengths, _slopes(c)


def _slopes(c):
    if not c["bias"]:
        return None
    h = c["q_heads"]
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32, device=DEV)


def _clip_inputs(c, seed):
    g = _generator(seed)
    # LoRA gradients differ by orders of magnitude between A and B and between layers
    grads = [_randn(g, s, t, 10.0 ** (-1 - 3 * ((7 * i) % 11) / 11.0))
             for i, (s, t) in enumerate(zip(_clip_shapes(c), _clip_dtypes(c)))]
    return grads, (1e-3 if c["clipped"] else 1e9)


def prepare(c, seed):
    st = {"case": c}
    if c["op"] == "rotary":
        q, k, dq, dk, pos = _rotary_inputs(c, seed)
        st.update(q=q, k=k, dq=dq, dk=dk, pos=pos)
        if own:
            import rank_linear_gb300 as rl
            st["freqs"] = rl.rotary_frequencies(c["rot"], base=ROTARY_BASE, scaling=SCALINGS[c["scaling"]], device=DEV)
        else:  # the plain form's program keeps a table of cosines and sines
            w, mag = _angular(c)
            n = c["far"] + c["seq"]
            a = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * torch.tensor(w, device=DEV, dtype=torch.float64)
            st["cos"], st["sin"] = (a.cos() * mag).float(), (a.sin() * mag).float()
    elif c["op"] == "attention":
        q, k, v, do, docs, prefix, slopes = _attention_inputs(c, seed)
        st.update(q=q, k=k, v=v, do=do, docs=docs, prefix=prefix, slopes=slopes)
    elif c["op"] == "decode":
        q, k, v, lengths, slopes = _decode_inputs(c, seed)
        st.update(q=q, k=k, v=v, lengths=lengths, slopes=slopes)
    else:
        grads, max_norm = _clip_inputs(c, seed)
        st.update(grads=grads, max_norm=max_norm)
        if own:  # the plan over the adapters' gradients, and the flat buffers that the optimiser reads
            import rank_linear_gb300 as rl
            kinds = sorted({t.dtype for t in grads}, key=str)
            st["out"] = [torch.empty(sum(t.numel() for t in grads if t.dtype == d), dtype=d, device=DEV) for d in kinds]
            parts = {d: iter(x.split([t.numel() for t in grads if t.dtype == d])) for d, x in zip(kinds, st["out"])}
            st["plan"] = rl.GradClip(grads, out=[next(parts[t.dtype]).view(t.shape) for t in grads])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    return (_run_own if own else _run_plain)[c["op"]](st, c)


def _own_rotary(st, c):
    import rank_linear_gb300 as rl
    out = rl.rotary_forward(st["q"], st["k"], st["pos"], st["freqs"], interleaved=c["interleaved"])
    if c["train"]:
        out += rl.rotary_backward(st["dq"], st["dk"], st["pos"], st["freqs"], interleaved=c["interleaved"])
    return out


def _own_attention(st, c):
    import rank_linear_gb300 as rl
    opts = dict(causal=c["causal"], softcap=c["cap"], slopes=st["slopes"], documents=st["docs"], prefix=st["prefix"])
    o, lse = rl.attention_forward(st["q"], st["k"], st["v"], **opts)
    if not c["train"]:
        return o
    return (o,) + rl.attention_backward(st["do"], st["q"], st["k"], st["v"], o, lse, **opts)


def _own_decode(st, c):
    import rank_linear_gb300 as rl
    return rl.attention_decode(st["q"], st["k"], st["v"], st["lengths"], softcap=c["cap"], slopes=st["slopes"])


def _own_clip(st, c):
    return [st["plan"].clip(st["max_norm"], norm_type=math.inf if c["largest"] else 2.0)] + st["out"]


_run_own = {"rotary": _own_rotary, "attention": _own_attention, "decode": _own_decode, "clip": _own_clip}


def _turn(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    f = x.float()
    a, b = (f[..., 0:r:2], f[..., 1:r:2]) if interleaved else (f[..., :r // 2], f[..., r // 2:r])
    u, w = a * cos - b * sin, b * cos + a * sin
    t = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((t, f[..., r:]), -1).to(x.dtype)


def _plain_rotary(st, c):
    cos, sin = st["cos"][st["pos"]][:, :, None], st["sin"][st["pos"]][:, :, None]
    i = c["interleaved"]
    out = (_turn(st["q"], cos, sin, i), _turn(st["k"], cos, sin, i))
    if c["train"]:
        out += (_turn(st["dq"], cos, -sin, i), _turn(st["dk"], cos, -sin, i))
    return out


def _mask(c, docs, prefix, device):
    """[batch, 1, 1, q, k]: what each query sees; None for everything."""
    sq, sk = c["q_len"], c["k_len"]
    m = None
    if c["causal"]:
        i = torch.arange(sq, device=device)[:, None] + (sk - sq)
        j = torch.arange(sk, device=device)[None]
        m = (j <= i)[None]
        if prefix is not None:
            m = m | (j[None] < prefix[:, None, None])
    if docs is not None:
        d = (docs[:, :, None] == docs[:, None, :]) & (docs[:, :, None] >= 0)
        m = d if m is None else m & d
    return None if m is None else m[:, None, None]


def _plain_attention(st, c):
    b, sq, sk, hq, hk, d = (c[n] for n in ("batch", "q_len", "k_len", "q_heads", "k_heads", "dim"))
    grp, cap, scale = hq // hk, c["cap"], d ** -0.5
    q = st["q"].float().view(b, sq, hk, grp, d).permute(0, 2, 3, 1, 4)
    k = st["k"].float().permute(0, 2, 1, 3)[:, :, None]
    v = st["v"].float().permute(0, 2, 1, 3)[:, :, None]
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    t = None
    if cap:
        t = torch.tanh(s.mul_(1.0 / cap))
        s = t * cap
    if st["slopes"] is not None:
        i = torch.arange(sq, device=q.device, dtype=torch.float32)[:, None] + float(sk - sq)
        far = (i - torch.arange(sk, device=q.device, dtype=torch.float32)[None]).abs()
        s -= st["slopes"].view(1, hk, grp, 1, 1) * far
    m = _mask(c, st["docs"], st["prefix"], q.device)
    if m is not None:
        s.masked_fill_(~m, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, 1.0, total)
    o = torch.matmul(p, v)
    back = lambda x: x.permute(0, 3, 1, 2, 4).reshape(b, sq, hq, d).to(torch.bfloat16)
    if not c["train"]:
        return back(o)
    do = st["do"].float().view(b, sq, hk, grp, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p, s
    if t is not None:
        ds -= ds * t * t
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2).mul_(scale)
    head = lambda x: x.permute(0, 2, 1, 3).contiguous().to(torch.bfloat16)
    return back(o), back(dq), head(dk), head(dv)


def _plain_decode(st, c):
    b, n, hq, hk, d = (c[x] for x in ("batch", "length", "q_heads", "k_heads", "dim"))
    q = st["q"].float().view(b, hk, hq // hk, d)
    k, v = st["k"].float().permute(0, 2, 1, 3), st["v"].float().permute(0, 2, 1, 3)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5)
    if c["cap"]:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    j = torch.arange(n, device=q.device)
    length = st["lengths"][:, None, None, None]
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, hk, hq // hk, 1) * (length - 1 - j).float()
    s = s.masked_fill(j >= length, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return o.view(b, hq, d).to(torch.bfloat16)


def _flat(grads, f):
    """f of every gradient, one flat tensor for each type."""
    return [torch.cat([f(t).flatten() for t in grads if t.dtype == d]) for d in sorted({t.dtype for t in grads}, key=str)]


def _plain_clip(st, c):
    if not c["largest"]:
        norm = torch.stack([t.float().square().sum() for t in st["grads"]]).sum().sqrt()
    else:
        norm = torch.stack([t.float().abs().max() for t in st["grads"]]).max()
    by = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    return [norm] + _flat(st["grads"], lambda t: (t.float() * by).to(t.dtype))


_run_plain = {"rotary": _plain_rotary, "attention": _plain_attention, "decode": _plain_decode, "clip": _plain_clip}


# ------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    return {"rotary": _exact_rotary, "attention": _exact_attention, "decode": _exact_decode, "clip": _exact_clip}[c["op"]](c, seed)


def _exact_rotary(c, seed):
    """Each pair as a complex number, turned by exp(i a)."""
    q, k, dq, dk, pos = _rotary_inputs(c, seed)
    w, mag = _angular(c)
    a = pos.double()[:, :, None, None] * torch.tensor(w, device=DEV, dtype=torch.float64)
    by = torch.polar(torch.full_like(a, mag), a)
    r = c["rot"]

    def turn(x, by):
        y = x.double()
        z = y[..., :r].unflatten(-1, (r // 2, 2) if c["interleaved"] else (2, r // 2))
        z = z if c["interleaved"] else z.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        out = y.clone()
        out[..., :r] = z.flatten(-2)
        return out

    out = (turn(q, by), turn(k, by))
    return out + (turn(dq, by.conj()), turn(dk, by.conj())) if c["train"] else out


def _exact_attention(c, seed):
    """Head by head, in blocks of queries; about 1e12 double operations take 2 s."""
    if 14 * c["dim"] * c["batch"] * c["q_heads"] * c["q_len"] * c["k_len"] > 6e12:
        return None
    q, k, v, do, docs, prefix, slopes = _attention_inputs(c, seed)
    b, sq, sk, hq, hk, d = (c[n] for n in ("batch", "q_len", "k_len", "q_heads", "k_heads", "dim"))
    o = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=DEV)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(b, sk, hk, d, dtype=torch.float64, device=DEV), None
    dv = torch.zeros_like(dk)
    key = torch.arange(sk, device=DEV)
    for n in range(b):
        for h in range(hq):
            g = h // (hq // hk)
            kk, vv = k[n, :, g].double(), v[n, :, g].double()
            for at in range(0, sq, 2048):
                rows = torch.arange(at, min(at + 2048, sq), device=DEV)
                place = rows + (sk - sq)
                qq = q[n, rows, h].double()
                z = qq @ kk.T / math.sqrt(d)
                u = torch.tanh(z / c["cap"]) if c["cap"] else None
                s = c["cap"] * u if c["cap"] else z
                if slopes is not None:
                    s = s - slopes[h].double() * (place[:, None] - key[None]).abs()
                see = torch.ones(len(rows), sk, dtype=torch.bool, device=DEV)
                if c["causal"]:
                    see = place[:, None] >= key[None]
                    if prefix is not None:
                        see = see | (key[None] < prefix[n])
                if docs is not None:
                    see = see & (docs[n, rows][:, None] == docs[n][None]) & (docs[n, rows][:, None] != -1)
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
                o[n, rows, h] = p @ vv
                if c["train"]:
                    e = do[n, rows, h].double()
                    dp = e @ vv.T
                    dz = p * (dp - (p * dp).sum(-1, keepdim=True))
                    if u is not None:
                        dz = dz * (1 - u * u)
                    dz = dz / math.sqrt(d)
                    dq[n, rows, h] = dz @ kk
                    dk[n, :, g] += dz.T @ qq
                    dv[n, :, g] += p.T @ e
    return (o, dq, dk, dv) if c["train"] else o


def _exact_decode(c, seed):
    q, k, v, lengths, slopes = _decode_inputs(c, seed)
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    grp = c["q_heads"] // c["k_heads"]
    for n, length in enumerate(_cache_lengths(c)):
        if length == 0:
            continue
        kk = k[n, :length].double().repeat_interleave(grp, 1)
        vv = v[n, :length].double().repeat_interleave(grp, 1)
        s = torch.einsum("hd,jhd->hj", q[n].double(), kk) / math.sqrt(c["dim"])
        if c["cap"]:
            s = c["cap"] * torch.tanh(s / c["cap"])
        if slopes is not None:
            s = s - slopes.double()[:, None] * torch.arange(length - 1, -1, -1, device=DEV)
        out[n] = torch.einsum("hj,jhd->hd", torch.softmax(s, -1), vv)
    return out


def _exact_clip(c, seed):
    grads, max_norm = _clip_inputs(c, seed)
    if not c["largest"]:
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in grads))
    else:
        norm = max(float(t.double().abs().max()) for t in grads)
    by = min(1.0, max_norm / (norm + 1e-6))
    return [torch.tensor(norm, dtype=torch.float64, device=DEV)] + _flat(grads, lambda t: t.double() * by)
