"""Cases of the operators before and after the LoRA layers of a step: the
root-mean-square norm with the residual's addition (and an 8-bit output),
dropout whose mask is generated again instead of stored, and the cross entropy
of a large vocabulary with its gradient.

Where `own` is false, `run` computes an operator from elementary torch
operations in 32 bits; where it is true, it calls this framework.  `exact`
gives the same outputs from the definitions in 64 bits.

Sizes: widths 4096 / 14336 are those of the framework's Llama-3-8B layers, 5120
that of its wide FFN workload, heads of 128 its attention's, a vocabulary of
128000 that of the loss the reference pages describe; the rest is generic.
"""
import math

import torch

own = False

DEV = "cuda:0"
BF16, FP32 = "bf16", "fp32"
TORCH = {BF16: torch.bfloat16, FP32: torch.float32}
SIZE = {BF16: 2, FP32: 4}
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # serving: the norm of one new token of 8 sequences, on the way to fp8 layers
        norm("norm_one_token", rows=8, heads=0, dim=4096, residual=True, p=0.0, fp8=True, train=False, dtype=BF16),
        # a training step: residual stream and norm before a block's first layers, forward and backward
        norm("norm_train", rows=8192, heads=0, dim=4096, residual=True, p=0.0, fp8=False, train=True, dtype=BF16),
        # the same with the branch dropped out before it joins the stream
        norm("norm_train_dropout", rows=16384, heads=0, dim=5120, residual=True, p=0.1, fp8=False, train=True, dtype=BF16),
        # a long prompt through the wide workload's norm, into fp8 layers
        norm("norm_prompt_fp8", rows=16384, heads=0, dim=5120, residual=True, p=0.0, fp8=True, train=False, dtype=BF16),
        # norms of every query head, read from a fused q|k|v output
        norm("norm_heads", rows=4096, heads=32, dim=128, residual=False, p=0.0, fp8=False, train=True, dtype=BF16),
        # an odd width in fp32
        norm("norm_odd_fp32", rows=5331, heads=0, dim=2001, residual=True, p=0.0, fp8=False, train=True, dtype=FP32),
        # a small odd tensor
        dropout("dropout_small", rows=514, dim=1001, p=0.5, train=True, dtype=BF16),
        # what goes into the down projection of a training step
        dropout("dropout_ffn", rows=8192, dim=14336, p=0.1, train=True, dtype=BF16),
        # serving: the log-probabilities of 8 tokens
        loss("loss_score_few", rows=8, dim=4096, vocab=128000, ignored=0.0, weighted=False, cap=0.0, train=False),
        # a short odd batch, half of it a prompt that does not count
        loss("loss_short_odd", rows=301, dim=1000, vocab=32003, ignored=0.5, weighted=False, cap=0.0, train=True),
        # capped logits and weighted tokens
        loss("loss_cap_weights", rows=2047, dim=5120, vocab=65537, ignored=0.1, weighted=True, cap=30.0, train=True),
        # a training step of 4 sequences of 2048 tokens
        loss("loss_train", rows=8192, dim=4096, vocab=128000, ignored=0.25, weighted=False, cap=0.0, train=True),
    ]


def norm(name=None, **kw):
    c = dict(op="norm", **kw)
    return {"name": name, **c} if name else c


def dropout(name=None, **kw):
    c = dict(op="dropout", **kw)
    return {"name": name, **c} if name else c


def loss(name=None, **kw):
    c = dict(op="loss", **kw)
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dropout", "loss", "loss"])
    dtype = rng.choice([BF16, BF16, FP32])
    if op == "norm":
        heads = rng.choice([0, 0, 0, 8, 32])
        if heads:
            dim = rng.choice([64, 80, 96, 128])
        else:
            dim = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024), 4096, 5120])
        size = 4 if dtype == FP32 else 2
        rows = _log_int(rng, 1, 160_000_000 // (size * dim * max(heads, 1)))
        fp8 = dtype == BF16 and not heads and rng.random() < 0.4
        residual = not heads and rng.random() < 0.7
        return norm(rows=rows, heads=heads, dim=dim, residual=residual,
                    p=rng.choice([0.0, 0.05, 0.3]) if residual else 0.0, fp8=fp8,
                    train=not fp8 and rng.random() < 0.7, dtype=dtype)
    if op == "dropout":
        dim = rng.choice([_log_int(rng, 1, 20000), 4096, 8 * _log_int(rng, 4, 2000)])
        return dropout(rows=_log_int(rng, 1, min(65536, (58_000_000 if dtype == FP32 else 117_000_000) // dim)), dim=dim,
                       p=rng.choice([0.01, 0.1, 0.25, 0.5, 0.9]), train=rng.random() < 0.6, dtype=dtype)
    dim = rng.choice([512, 1000, 2048, 4096, 5120])
    vocab = _log_int(rng, 1000, min(160000, 520_000_000 // dim))
    # at most the listed cases' work
    rows = _log_int(rng, 1, min(16384, int(3.2e12 / (dim * vocab))))
    return loss(rows=rows, dim=dim, vocab=vocab, ignored=rng.choice([0.0, 0.3, 0.8]),
                weighted=rng.random() < 0.3, cap=rng.choice([0.0, 0.0, 30.0]), train=rng.random() < 0.7)


# ------------------------------------------------------------------ work

def work(c):
    if c["op"] == "norm":
        n = c["rows"] * max(c["heads"], 1) * c["dim"]
        s = SIZE[c["dtype"]]
        # x (and the residual) in, y (and the sum) out
        moved = (4 if c["residual"] else 2) * n * s + (n if c["fp8"] else 0)
        flops = 5 * n
        if c["train"]:  # dy, the normed input (and the stream's gradient) in, dx (two, where one is dropped out) out
            moved += (3 + (1 if c["residual"] else 0) + (1 if c["p"] else 0)) * n * s
            flops += 10 * n
        return {"bytes": moved, "flops": flops}
    if c["op"] == "dropout":
        n = c["rows"] * c["dim"] * (2 if c["train"] else 1)
        return {"bytes": 2 * n * SIZE[c["dtype"]], "flops": n}
    n, d, v = c["rows"], c["dim"], c["vocab"]
    live = n - len(_ignored_rows(c))
    return {"bytes": v * d * 2 + live * d * (4 if c["train"] else 2) + n * 12,
            "flops": 2 * live * d * v * (2 if c["train"] else 1)}


def _ignored_rows(c):
    """Runs of tokens that do not count, as prompts in front of answers: four of them."""
    n, out = c["rows"], []
    for i in range(4):
        a, b = n * i // 4, n * (i + 1) // 4
        out += range(a, a + int(round((b - a) * c["ignored"])))
    return out


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(TORCH[dtype])


def _norm_inputs(c, seed):
    g = _generator(seed)
    n, d, t = c["rows"], c["dim"], c["dtype"]
    if c["heads"]:  # the query heads of a fused q|k|v output: a strided view
        shape = (n, c["heads"], d)
        x = _randn(g, (n, c["heads"] + c["heads"] // 2, d), t, 2.0)[:, :c["heads"]]
    else:
        shape = (n, d)
        x = _randn(g, shape, t)
    res = _randn(g, shape, t, 3.0) if c["residual"] else None
    w = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(TORCH[t])
    dy = dh = None
    if c["train"]:
        dy = _randn(g, shape, t, 0.1)
        dh = _randn(g, shape, t, 0.1) if c["residual"] else None
    return x, res, w, dy, dh


def _dropout_inputs(c, seed):
    g = _generator(seed)
    x = _randn(g, (c["rows"], c["dim"]), c["dtype"])
    return x, (_randn(g, (c["rows"], c["dim"]), c["dtype"]) if c["train"] else None)


def _loss_inputs(c, seed):
    g = _generator(seed)
    n, d, v = c["rows"], c["dim"], c["vocab"]
    w = _randn(g, (v, d), BF16, 2.0 * d ** -0.5)
    targets = torch.randint(0, v, (n,), generator=g, device=DEV)
    # a trained model's hidden states lean towards the token that comes next: losses from nearly 0 to 12
    x = torch.randn(n, d, generator=g, device=DEV)
    x = (x + 3.5 * torch.rand(n, 1, generator=g, device=DEV) * w[targets].float()).bfloat16()
    weights = torch.rand(n, generator=g, device=DEV) if c["weighted"] else None
    skip = _ignored_rows(c)
    if skip:
        targets[torch.tensor(skip, device=DEV)] = -100
    return x, w, targets, weights


def _mask_key(seed):
    """(seed, offset) of a case's dropout."""
    return 0x9E3779B97F4A7C15 * (seed + 1) % 2 ** 63, 7 + seed % 1000


def prepare(c, seed):
    st = {"case": c, "key": _mask_key(seed)}
    if c["op"] == "norm":
        st.update(zip(("x", "res", "w", "dy", "dh"), _norm_inputs(c, seed)))
    elif c["op"] == "dropout":
        st.update(zip(("x", "dy"), _dropout_inputs(c, seed)))
    else:
        st.update(zip(("x", "w", "targets", "weights"), _loss_inputs(c, seed)))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    return (_run_own if own else _run_plain)[c["op"]](st, c)


def _own_norm(st, c):
    import rank_linear_gb300 as rl
    seed, offset = st["key"]
    drop = dict(dropout=c["p"], seed=seed, offset=offset)
    if c["fp8"]:
        y, h, _, codes, scale = rl.rms_norm_forward(st["x"], st["w"], residual=st["res"], eps=EPS, fp8=True, **drop)
        out = [y, codes.view(torch.float8_e4m3fn), scale]
    else:
        y, h, rstd = rl.rms_norm_forward(st["x"], st["w"], residual=st["res"], eps=EPS, **drop)
        out = [y]
    if c["residual"]:
        out.append(h)
    if c["train"]:
        dx, dres, dw = rl.rms_norm_backward(st["dy"], h, st["w"], rstd, dh=st["dh"], **drop)
        out += [dx, dw] + ([dres] if c["p"] else [])
    return out


def _own_dropout(st, c):
    import rank_linear_gb300 as rl
    seed, offset = st["key"]
    y = rl.dropout_forward(st["x"], c["p"], seed, offset)
    return (y, rl.dropout_backward(st["dy"], c["p"], seed, offset)) if c["train"] else y


def _own_loss(st, c):
    import rank_linear_gb300 as rl
    mean, each, dx = rl.cross_entropy_forward(st["x"], st["w"], st["targets"], weights=st["weights"],
                                              softcap=c["cap"], gradient=c["train"])
    return (mean, each, dx) if c["train"] else (mean, each)


_run_own = {"norm": _own_norm, "dropout": _own_dropout, "loss": _own_loss}

LOW = 0xFFFFFFFF


def _random_words(rows, dim, key):
    """[rows, dim] words in 0 .. 2^32 - 1: Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
    random numbers: as easy as 1, 2, 3", 2011), key = the seed, counter = (column // 4, row, row >> 32, offset)."""
    seed, offset = key
    blocks = (dim + 3) // 4
    row = torch.arange(rows, device=DEV)[:, None].expand(rows, blocks)
    a = torch.arange(blocks, device=DEV)[None].expand(rows, blocks)
    b, c, d = row & LOW, row >> 32, torch.full_like(row, offset)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((q >> 32) & LOW) ^ b ^ k0, q & LOW, ((p >> 32) & LOW) ^ d ^ k1, p & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack((a, b, c, d), -1).flatten(1)[:, :dim]


def _drop_threshold(p):
    return int(round(p * 2 ** 32))


def _drop32(x, p, key):
    t = _drop_threshold(p)
    return torch.where(_random_words(*x.shape, key) >= t, x * (2.0 ** 32 / (2 ** 32 - t)), 0.0)


def _plain_norm(st, c):
    x, w = st["x"].float(), st["w"].float()
    h = x
    if c["residual"]:
        h = (_drop32(x, c["p"], st["key"]) if c["p"] else x) + st["res"].float()
        h = h.to(TORCH[c["dtype"]])  # the stream that the next block adds to: the norm is of what it holds
        stream, h = h, h.float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    y = h * r * w
    out = [y.to(TORCH[c["dtype"]])]
    if c["fp8"]:
        top = y.abs().amax(-1, keepdim=True)
        m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
        e = torch.where(top > 0, e - 8 - (m <= 0.875).int(), 0)
        scale = torch.ldexp(torch.ones_like(top), e)
        out += [(y / scale).to(torch.float8_e4m3fn), scale[:, 0]]
    if c["residual"]:
        out.append(stream)
    if c["train"]:
        dy = st["dy"].float()
        hat = h * r
        g = dy * w
        dh = r * (g - hat * (g * hat).mean(-1, keepdim=True))
        if st["dh"] is not None:
            dh = dh + st["dh"].float()
        dw = (dy * hat).flatten(0, -2).sum(0).to(st["w"].dtype)
        if c["p"]:
            out += [_drop32(dh, c["p"], st["key"]).to(TORCH[c["dtype"]]), dw, dh.to(TORCH[c["dtype"]])]
        else:
            out += [dh.to(TORCH[c["dtype"]]), dw]
    return out


def _plain_dropout(st, c):
    y = _drop32(st["x"].float(), c["p"], st["key"]).to(TORCH[c["dtype"]])
    return (y, _drop32(st["dy"].float(), c["p"], st["key"]).to(TORCH[c["dtype"]])) if c["train"] else y


def _plain_loss(st, c):
    x, w, targets, cap = st["x"].float(), st["w"].float(), st["targets"], c["cap"]
    counts = (targets >= 0).float()
    if st["weights"] is not None:
        counts = counts * st["weights"]
    total = counts.sum()
    g = counts / torch.where(total == 0, 1.0, total)
    each, dx = [], []
    for at in range(0, c["rows"], 2048):  # in pieces, as the logits of all rows would take gigabytes
        rows = slice(at, at + 2048)
        z = torch.matmul(x[rows], w.T)
        t = None
        if cap:
            t = torch.tanh(z.mul_(1.0 / cap))
            z = t * cap
        to = targets[rows].clamp(min=0)[:, None]
        z_to = z.gather(1, to)
        top = z.amax(-1, keepdim=True)
        p = (z - top).exp_()
        s = p.sum(-1, keepdim=True)
        each.append(torch.where(targets[rows] >= 0, (s.log() + top - z_to)[:, 0], 0.0))
        if c["train"]:
            p /= s
            p.scatter_add_(1, to, torch.full_like(z_to, -1.0))
            if cap:
                p *= 1.0 - t * t
            dx.append((torch.matmul(p, w) * g[rows, None]).to(torch.bfloat16))
    each = torch.cat(each)
    mean = (each * g).sum()
    return (mean, each, torch.cat(dx)) if c["train"] else (mean, each)


_run_plain = {"norm": _plain_norm, "dropout": _plain_dropout, "loss": _plain_loss}


# ------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    return {"norm": _exact_norm, "dropout": _exact_dropout, "loss": _exact_loss}[c["op"]](c, seed)


def _kept(rows, dim, p, key):
    """[rows, dim] truth values: the generator again, its products from halves of 16 bits."""
    def product(u, m):
        lo, hi = u * (m & 0xFFFF), u * (m >> 16)
        mid = (lo >> 16) + (hi & 0xFFFF)
        return (hi >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)

    column = torch.arange((dim + 3) // 4, device=DEV)
    out = torch.empty(rows, dim, dtype=torch.bool, device=DEV)
    step = max(1, 2 ** 24 // len(column))
    for at in range(0, rows, step):
        row = torch.arange(at, min(at + step, rows), device=DEV)
        x = [column.expand(len(row), -1), (row % 2 ** 32)[:, None].expand(-1, len(column)),
             (row // 2 ** 32)[:, None].expand(-1, len(column)), torch.full((len(row), len(column)), key[1], device=DEV)]
        for i in range(10):
            k0 = (key[0] % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32
            k1 = (key[0] // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
            h0, l0 = product(x[0], 0xD2511F53)
            h2, l2 = product(x[2], 0xCD9E8D57)
            x = [h2 ^ x[1] ^ k0, l2, h0 ^ x[3] ^ k1, l0]
        for j in range(4):
            n = len(range(j, dim, 4))
            out[at:at + step, j::4] = x[j][:, :n] >= _drop_threshold(p)
    return out


def _exact_drop(x, p, key):
    keep = 1.0 - _drop_threshold(p) / 2.0 ** 32
    return torch.where(_kept(*x.shape, p, key), x.double() / keep, torch.zeros((), dtype=torch.float64, device=DEV))


def _exact_norm(c, seed):
    x, res, w, dy, dh = _norm_inputs(c, seed)
    key = _mask_key(seed)
    h = x.double()
    if c["p"]:
        h = _exact_drop(x, c["p"], key)
    if res is not None:
        # held as the inputs' type, rounded once; the norm is of what is held
        stream = h + res.double()
        h = stream.to(x.dtype).double()
    norm2 = torch.linalg.vector_norm(h, dim=-1, keepdim=True)
    length = torch.sqrt(norm2 * norm2 / c["dim"] + EPS)
    unit = h / length
    y = unit * w.double()
    out = [y]
    if c["fp8"]:
        top = y.abs().amax(-1)
        scale = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / 448.0))), 1.0)
        out += [y / scale[:, None], scale]
    if res is not None:
        out.append(stream)
    if c["train"]:
        along = dy.double() * w.double()
        dh_all = (along - unit * torch.einsum("...d,...d->...", along, unit)[..., None] / c["dim"]) / length
        if dh is not None:
            dh_all = dh_all + dh.double()
        dw = torch.einsum("...d,...d->d", dy.double(), unit)
        if c["p"]:
            out += [_exact_drop(dh_all, c["p"], key), dw, dh_all]
        else:
            out += [dh_all, dw]
    return out


def _exact_dropout(c, seed):
    x, dy = _dropout_inputs(c, seed)
    y = _exact_drop(x, c["p"], _mask_key(seed))
    return (y, _exact_drop(dy, c["p"], _mask_key(seed))) if c["train"] else y


def _exact_loss(c, seed):
    """About 1e12 double operations take a second."""
    if 4 * c["rows"] * c["dim"] * c["vocab"] > 8e12:
        return None
    x, w, targets, weights = _loss_inputs(c, seed)
    w = w.double()
    share = (targets != -100).double()
    if weights is not None:
        share = share * weights.double()
    share = share / max(float(share.sum()), 1e-300)
    each = torch.zeros(c["rows"], dtype=torch.float64, device=DEV)
    dx = torch.zeros(c["rows"], c["dim"], dtype=torch.float64, device=DEV)
    live = torch.nonzero(targets != -100)[:, 0]
    for rows in live.split(1024):
        raw = x[rows].double() @ w.T
        z = c["cap"] * torch.tanh(raw / c["cap"]) if c["cap"] else raw
        at = torch.arange(len(rows), device=DEV)
        logp = z - torch.logsumexp(z, -1, keepdim=True)
        each[rows] = -logp[at, targets[rows]]
        if c["train"]:
            dz = torch.exp(logp)
            dz[at, targets[rows]] = torch.expm1(logp[at, targets[rows]])
            if c["cap"]:
                dz = dz * torch.cosh(raw / c["cap"]) ** -2
            dx[rows] = (dz * share[rows, None]) @ w
    mean = torch.dot(each, share)
    return (mean, each, dx) if c["train"] else (mean, each)
