"""Masked attention on the GPU against its definition in 64 bits (needs a GB300).

Every element of o, dq, dk and dv has to lie within the forward-error bound of
its bf16 form (oracle.attention.run): P and dz are rounded to bf16 once (2^-8
relative each), an output once more, and what is computed in fp32 adds less
than 2^-11; sums carry those errors through absolute values.  lse: fp32, 2^-14
of its magnitude plus 2^-11.
"""
import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import attention as oa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TINY = 1e-30


def draw(B, sq, sk, hq, hk, d, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return (r(B, sq, hq, d) * gain).bfloat16(), r(B, sk, hk, d).bfloat16(), \
        r(B, sk, hk, d).bfloat16(), r(B, sq, hq, d).bfloat16()


def host(t):
    return None if t is None else t.double().numpy() if t.is_floating_point() else t.numpy()


def compare(got, ref, names):
    for n in names:
        a = got[n].double().cpu().numpy()
        if n == "lse":
            r = ref["lse"]
            assert np.array_equal(np.isneginf(a), np.isneginf(r)), "lse of empty rows"
            fin = np.isfinite(r)
            assert np.all(np.abs(a - r)[fin] <= 2 ** -14 * np.abs(r[fin]) + 2 ** -11)
            continue
        assert np.isfinite(a).all(), f"{n} is not finite"
        err, bound = np.abs(a - ref[n]), ref["bound"][n] + TINY
        if not err.size:
            continue
        worst = np.unravel_index(np.argmax(err - bound), err.shape)
        assert np.all(err <= bound), f"{n}{worst}: {a[worst]} against {ref[n][worst]}, bound {bound[worst]}"


def check(q, k, v, do, *, causal=False, cap=0.0, slopes=None, prefix=None, docs=None, scale=None,
          backward=True):
    dev = lambda t: None if t is None else t.to(DEV)
    pair = isinstance(docs, tuple)
    qd, kd = docs if pair else (docs, docs)
    if docs is not None and not pair and q.shape[1] != k.shape[1]:
        qd = docs[:, k.shape[1] - q.shape[1]:]
    opts = dict(causal=causal, softcap=cap, slopes=dev(slopes), prefix=dev(prefix), scale=scale,
                documents=tuple(map(dev, docs)) if pair else dev(docs))
    gq, gk, gv, gdo = map(dev, (q, k, v, do))
    o, lse = rl.attention_forward(gq, gk, gv, **opts)
    got = dict(o=o, lse=lse)
    names = ["o", "lse"]
    if backward:
        got["dq"], got["dk"], got["dv"] = rl.attention_backward(gdo, gq, gk, gv, o, lse, **opts)
        names += ["dq", "dk", "dv"]
    torch.cuda.synchronize()
    rl.device_status()
    ref = oa.run(host(q), host(k), host(v), host(do) if backward else None,
                 scale=q.shape[-1] ** -0.5 if scale is None else scale, causal=causal, cap=cap,
                 slopes=host(slopes), prefix=host(prefix), q_docs=host(qd), k_docs=host(kd))
    compare(got, ref, names)
    return got


def slopes_of(h):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("sq,sk", [(1, 1), (2, 3), (127, 127), (128, 128), (129, 129), (255, 300),
                                   (257, 513), (1, 700), (64, 640), (384, 384)])
def test_lengths(sq, sk, causal):
    check(*draw(1, sq, sk, 4, 2, 64, sq * 1000 + sk), causal=causal)


@pytest.mark.parametrize("d", [8, 16, 40, 64, 72, 96, 120, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_head_sizes(d, cap):
    check(*draw(2, 200, 200, 2, 1, d, d, gain=3.0 if cap else 1.0), causal=True, cap=cap)


@pytest.mark.parametrize("cap", [1.5, 4.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_beyond_the_cap(d, cap):
    """Most tiles have a score above the cap, some (quiet keys) have none."""
    q, k, v, do = draw(2, 390, 390, 4, 2, d, 40, gain=2.0)
    k[:, 128:256] *= 0.1
    check(q, k, v, do, causal=True, cap=cap)
    check(q, k, v, do, cap=cap, slopes=slopes_of(4))


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 8), (8, 1), (10, 2), (40, 8)])
def test_head_groups(hq, hk):
    check(*draw(2, 150, 150, hq, hk, 128 if hq < 10 else 64, hq), causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cap", [0.0, 15.0])
@pytest.mark.parametrize("d", [64, 128])
def test_distance_bias(causal, cap, d):
    check(*draw(1, 300, 300, 4, 2, d, 5, gain=3.0 if cap else 1.0), causal=causal, cap=cap,
          slopes=slopes_of(4))
    check(*draw(1, 130, 300, 4, 2, d, 6), causal=causal, slopes=slopes_of(4))


@pytest.mark.parametrize("n", [0, 1, 64, 128, 200, 299, 300, 5000])
def test_prefix(n):
    p = torch.tensor([n, max(0, n - 1)], dtype=torch.int32)
    check(*draw(2, 300, 300, 2, 1, 64, n), causal=True, prefix=p)
    check(*draw(2, 50, 300, 2, 1, 128, n + 1), causal=True, prefix=p)


def packed(lengths, pad, B=1):
    row = sum(([i] * n for i, n in enumerate(lengths)), []) + [-1] * pad
    return torch.tensor([row] * B, dtype=torch.int32)


def few_keys(gpu, q, k, v, do, cap=0.0, causal=True, docs=None):
    """dq and dk where delta is not taken from the rounded o.  Sums over at most
    128 products in fp32 are off by 2^-16 of their terms' magnitude (128
    roundings of 2^-24, twice that where the tensor cores truncate), scores of
    sum |q k| scale <= 24 by 24 * 2^-17, hence P by less than 2^-12 of itself
    (the exponential and the cap add 2^-20).  dz = P (dP - delta), delta the
    sum of the same P dP, is then off by 2^-12 P (|dP| + sum P |dP|) and the
    error of dP, and is rounded to bf16 once, as its sums are."""
    G, M = 2.0 ** -12, 2.0 ** -16
    scale = q.shape[-1] ** -0.5
    for b in range(q.shape[0]):
        see = oa.visible(q.shape[1], k.shape[1], causal, 0, *((None, None) if docs is None else (docs[b],) * 2))
        for g in range(k.shape[2]):
            dk, dkb = 0.0, TINY
            for h in range(g * (q.shape[2] // k.shape[2]), (g + 1) * (q.shape[2] // k.shape[2])):
                p, sl, o, _, qkv = oa.head(q[b, :, h], k[b, :, g], v[b, :, g], scale=scale, see=see, cap=cap)
                grad = oa.head_backward(do[b, :, h], p, sl, o, qkv, scale=scale, see=see)
                dp = np.abs(grad[4] @ qkv[2].T)
                size = np.abs(grad[4]) @ np.abs(qkv[2]).T
                off = p * sl * (G * (dp + (p * dp).sum(1, keepdims=True)) + M * (size + (p * size).sum(1, keepdims=True)))
                dz = 2 * oa.U * np.abs(grad[3]) + off
                err = np.abs(gpu["dq"][b, :, h].double().cpu().numpy() - grad[0])
                assert np.all(err <= scale * dz @ np.abs(qkv[1]) + TINY), ("dq", b, h, err.max())
                dk, dkb = dk + grad[1], dkb + scale * dz.T @ np.abs(qkv[0])
            err = np.abs(gpu["dk"][b, :, g].double().cpu().numpy() - dk)
            assert np.all(err <= dkb), ("dk", b, g, err.max())


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("sq,sk,d,causal", [(2, 2, 128, True), (2, 2, 80, False), (3, 3, 96, True), (8, 8, 64, True),
                                            (100, 100, 128, True), (128, 128, 64, True), (300, 128, 128, False),
                                            (37, 125, 64, True)])
def test_gradients_that_nearly_cancel(sq, sk, d, causal, cap):
    """Few keys, a query that looks almost wholly at one of them."""
    q, k, v, do = draw(2, sq, sk, 8, 2, d, sq + sk + d)
    k[:, 0] *= 3  # the first key draws most of its queries' weight, or none
    got = check(q, k, v, do, causal=causal, cap=cap)
    few_keys(got, host(q), host(k), host(v), host(do), cap, causal)


def test_few_keys_and_padding():
    q, k, v, do = draw(1, 90, 90, 4, 2, 64, 9)
    docs = torch.tensor([[0] * 40 + [1] * 1 + [2] * 2 + [3] * 30 + [-1] * 17], dtype=torch.int32)
    for t in (q, k, v, do):
        t[:, -17:] = float("nan")
    got = check(q, k, v, do, causal=True, docs=docs)
    zero = [t.nan_to_num(0.0) for t in (q, k, v, do)]
    few_keys(got, *map(host, zero), docs=host(docs))
    for n in ("dq", "dk", "dv"):
        assert not got[n][:, -17:].any(), n


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths,pad", [([300], 0), ([128, 128, 256], 0), ([1, 127, 130, 42], 0),
                                         ([5] * 60, 0), ([100, 200], 84), ([1], 399), ([], 300)])
def test_packed_documents(lengths, pad, causal):
    docs = packed(lengths, pad, 2)
    n = docs.shape[1]
    check(*draw(2, n, n, 4, 2, 64, n), causal=causal, docs=docs)
    check(*draw(2, n, n, 2, 2, 128, n), causal=causal, docs=docs)


def test_documents_in_any_order():
    g = torch.Generator().manual_seed(3)
    docs = torch.randint(-1, 4, (2, 400), generator=g, dtype=torch.int32)
    check(*draw(2, 400, 400, 2, 1, 128, 3), causal=True, docs=docs)
    check(*draw(2, 400, 400, 2, 1, 64, 4), docs=docs, slopes=slopes_of(2))
    check(*draw(2, 150, 400, 2, 1, 64, 4), docs=docs, causal=True,
          prefix=torch.tensor([90, 390], dtype=torch.int32))
    qd = torch.randint(-1, 4, (2, 90), generator=g, dtype=torch.int32)
    check(*draw(2, 90, 400, 2, 1, 64, 4), docs=(qd, docs))


@pytest.mark.parametrize("sq,sk", [(300, 100), (200, 1), (130, 0), (129, 128)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(sq, sk, d):
    got = check(*draw(1, sq, sk, 2, 1, d, 1), causal=True)
    assert (got["o"][:, :sq - sk] == 0).all() and (got["dq"][:, :sq - sk] == 0).all()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 3.38e38])
@pytest.mark.parametrize("d", [64, 128])
def test_what_padding_holds_reaches_nothing(fill, d):
    docs = packed([70, 150, 60], 120)
    docs[0, 30:40] = -1
    q, k, v, do = draw(1, 400, 400, 4, 2, d, 8)
    for t in (q, k, v, do):
        t[docs < 0] = fill
    got = check(q, k, v, do, causal=True, docs=docs)
    for n in ("o", "dq", "dk", "dv"):
        assert (got[n].cpu()[docs < 0] == 0).all(), n


def test_masked_scores_are_replaced():
    """Infinite and lowest scores in masked places (future keys with huge k)."""
    q, k, v, do = draw(1, 260, 260, 2, 2, 64, 9)
    k[:, 200:] = torch.finfo(torch.bfloat16).max
    q[:, 200:] = 0
    check(q, k, v, do, causal=True, backward=False)


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (4, 4, 64), (6, 2, 96)])
def test_views_of_one_fused_tensor(hq, hk, d):
    """q, k and v as strided views of a q|k|v output, gradients into a fused buffer."""
    B, n = 2, 260
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, n, hq + 2 * hk, d, generator=g).bfloat16()
    do = torch.randn(n, B, d, hq, generator=g).bfloat16().permute(1, 0, 3, 2).contiguous()
    ref = oa.run(*(t.double().numpy() for t in x.split([hq, hk, hk], 2)), do.double().numpy(),
                 scale=d ** -0.5, causal=True)
    gx = x.to(DEV)
    q, k, v = gx.split([hq, hk, hk], 2)
    # o and do as [batch, heads, len, dim] seen through a transpose
    out = torch.empty(B, hq, n, d, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    gdo = do.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    o, lse = rl.attention_forward(q, k, v, causal=True, out=out)
    dx = torch.full_like(gx, float("nan"))
    dq, dk, dv = dx.split([hq, hk, hk], 2)
    rl.attention_backward(gdo, q, k, v, o, lse, causal=True, dq=dq, dk=dk, dv=dv)
    assert o is out
    compare(dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv), ref, ["o", "lse", "dq", "dk", "dv"])


def test_long_and_ragged():
    check(*draw(1, 1111, 1777, 3, 1, 128, 2), causal=True)
    check(*draw(1, 1500, 1500, 2, 1, 64, 2), cap=30.0)


def test_large_scores():
    """Scores far apart: the running maximum moves by hundreds."""
    q, k, v, do = draw(1, 400, 400, 2, 1, 64, 12)
    k *= torch.linspace(0.1, 4, 400)[None, :, None, None].bfloat16()
    check(q, k, v, do, causal=False, backward=False)
    k = k.flip(1)
    check(q, k, v, do, causal=False, backward=False)


CUT = [
    # batch, q_len, k_len, q_heads, k_heads, dim, causal: few queries over many keys
    (1, 1, 5000, 8, 2, 64, True), (2, 17, 4999, 4, 1, 128, True), (1, 300, 6000, 4, 2, 128, True),
    (3, 129, 3333, 2, 2, 80, False), (1, 255, 20001, 1, 1, 128, True), (1, 2048, 2048, 1, 1, 128, True),
    (5, 256, 2500, 8, 4, 40, False),
    # more items than blocks: the last round's are cut
    (1, 1025, 5100, 40, 8, 16, True), (2, 600, 6001, 27, 27, 8, False),
]


@pytest.mark.parametrize("B,sq,sk,hq,hk,d,causal", CUT)
def test_few_items_are_cut_along_the_keys(B, sq, sk, hq, hk, d, causal):
    q, k, v, do = draw(B, sq, sk, hq, hk, d, sk)
    before = rl.launch_count()
    check(q, k, v, do, causal=causal, backward=False)
    assert rl.launch_count() == before + 2, "attention and a join"


@pytest.mark.parametrize("hq,hk,sq", [(8, 1, 32), (8, 1, 33), (16, 2, 16), (4, 2, 64), (4, 2, 65), (4, 2, 128),
                                      (12, 1, 20), (12, 2, 100), (5, 1, 7), (64, 1, 3), (128, 1, 1), (24, 3, 31)])
@pytest.mark.parametrize("sk", [130, 3000])
def test_heads_of_a_group_side_by_side(hq, hk, sq, sk):
    """Few queries, alone and cut along the keys; full and ragged tiles."""
    d = 64 if sk > 1000 else 128
    q, k, v, do = draw(2, sq, sk, hq, hk, d, hq * sq)
    check(q, k, v, do, causal=True, slopes=slopes_of(hq), backward=sk < 1000)
    check(q, k, v, do, causal=True, cap=8.0, prefix=torch.tensor([sk // 2, 0], dtype=torch.int32),
          backward=False)
    docs = torch.arange(sk, dtype=torch.int32)[None].repeat(2, 1) // 50
    docs[1, -sq:] = torch.arange(sq, dtype=torch.int32) % 3 - 1 + sk // 50 - 2
    check(q, k, v, do, docs=docs, backward=False)
    # q is a view of a fused q|k|v output, o is given with strides of its own
    wide = torch.randn(2, sq, hq + 2, d).bfloat16()
    wide[:, :, 1:-1] = q
    dev = wide.to(DEV)[:, :, 1:-1]
    out = torch.full((2, sq, hq + 1, 2 * d), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse = rl.attention_forward(dev, k.to(DEV), v.to(DEV), out=out[:, :, :hq, :d])
    want, lse1 = rl.attention_forward(q.to(DEV), k.to(DEV), v.to(DEV))
    assert torch.equal(o, want) and torch.equal(lse, lse1)
    assert bool((out[:, :, hq:] == 7).all()) and bool((out[..., d:] == 7).all())


def test_cut_items_with_every_score_and_mask():
    q, k, v, do = draw(2, 200, 4100, 4, 2, 64, 5, gain=2.0)
    check(q, k, v, do, causal=True, cap=5.0, backward=False)
    check(q, k, v, do, causal=True, slopes=slopes_of(4), backward=False)
    check(q, k, v, do, causal=True, prefix=torch.tensor([0, 4000], dtype=torch.int32), backward=False)
    # documents: rows whose keys lie in one part only, in several, or nowhere
    docs = packed([1000, 2500, 17, 33, 400, 50], 100, 2)
    docs[1, :3000] = 7
    check(q, k, v, do, causal=True, docs=docs, backward=False)
    qd = torch.full((2, 200), 5, dtype=torch.int32)
    qd[:, 50:] = 3
    check(q, k, v, do, docs=(qd, docs), backward=False)
    # the gradients take the joined lse
    check(q[:, :, :2], k[:, :, :1], v[:, :, :1], do[:, :, :2], causal=True, cap=30.0)


@pytest.mark.parametrize("shape", [(1, 300, 6000, 4, 2, 128), (1, 1025, 5100, 40, 8, 16)])
def test_cut_items_repeat_bit_for_bit(shape):
    q, k, v, _ = (t.to(DEV) for t in draw(*shape, 3))
    o, lse = rl.attention_forward(q, k, v, causal=True)
    for _ in range(3):
        o1, lse1 = rl.attention_forward(q, k, v, causal=True)
        assert torch.equal(o, o1) and torch.equal(lse, lse1)


@pytest.mark.parametrize("sk", [300, 6000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_shows(sk, bad):
    """A query that is not finite makes its own row NaN, and no other one; a key
    every row that sees it."""
    q, k, v, do = (t.to(DEV) for t in draw(1, 200, sk, 2, 1, 64, 8))
    o, lse = rl.attention_forward(q, k, v)
    dq = rl.attention_backward(do, q, k, v, o, lse)[0]
    q[0, 77, 1, 3] = bad
    o1, lse1 = rl.attention_forward(q, k, v)
    dq1 = rl.attention_backward(do, q, k, v, o1, lse1)[0]
    assert o1[0, 77, 1].isnan().all() and lse1[0, 1, 77].isnan() and dq1[0, 77, 1].isnan().all()
    for clean, other in ((o, o1), (dq, dq1), (lse.transpose(1, 2), lse1.transpose(1, 2))):
        other[0, 77, 1] = clean[0, 77, 1]
        assert torch.equal(clean, other)
    k[0, 250] = float("nan")
    assert rl.attention_forward(q, k, v)[0].isnan().all()
    n = torch.tensor([sk], dtype=torch.int32, device=DEV)
    assert rl.attention_decode(q[:, 0], k, v, n).isnan().all()


def test_same_bits_each_time():
    q, k, v, do = (t.to(DEV) for t in draw(2, 700, 700, 8, 2, 128, 4))
    runs = []
    for _ in range(3):
        o, lse = rl.attention_forward(q, k, v, causal=True)
        runs.append((o, lse) + rl.attention_backward(do, q, k, v, o, lse, causal=True))
    for a, b in zip(runs[0], runs[1]):
        assert torch.equal(a, b)
    for a, b in zip(runs[0], runs[2]):
        assert torch.equal(a, b)


def test_on_another_stream():
    q, k, v, do = draw(1, 333, 333, 4, 2, 64, 7)
    s = torch.cuda.Stream()
    gq, gk, gv, gdo = (t.to(DEV) for t in (q, k, v, do))
    torch.cuda.synchronize()
    o, lse = rl.attention_forward(gq, gk, gv, causal=True, stream=s)
    grads = rl.attention_backward(gdo, gq, gk, gv, o, lse, causal=True, stream=s)
    s.synchronize()
    ref = oa.run(*map(host, (q, k, v, do)), scale=64 ** -0.5, causal=True)
    compare(dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads)), ref,
            ["o", "lse", "dq", "dk", "dv"])


def test_inside_a_graph():
    q, k, v, do = draw(1, 200, 200, 4, 2, 128, 17)
    gq, gk, gv, gdo = (t.to(DEV) for t in (q, k, v, do))
    rl.attention_forward(gq, gk, gv, causal=True)  # first calls outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = rl.attention_forward(gq, gk, gv, causal=True)
        grads = rl.attention_backward(gdo, gq, gk, gv, o, lse, causal=True)
    for t in (o, lse) + grads:
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    ref = oa.run(*map(host, (q, k, v, do)), scale=128 ** -0.5, causal=True)
    compare(dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads)), ref,
            ["o", "lse", "dq", "dk", "dv"])


def test_autograd():
    q, k, v, do = draw(2, 140, 140, 6, 3, 64, 21)
    ref = oa.run(*map(host, (q, k, v, do)), scale=0.1, causal=True, cap=25.0)
    x = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    o = rl.attention(*x, causal=True, softcap=25.0, scale=0.1)
    o.backward(do.to(DEV))
    compare(dict(o=o.detach(), dq=x[0].grad, dk=x[1].grad, dv=x[2].grad), ref,
            ["o", "dq", "dk", "dv"])


@pytest.mark.parametrize("cap", [0.0, 10.0])
def test_gradients_against_differences(cap):
    """<gradient, direction> against the central difference of the loss
    sum(o * do) in 64 bits; the difference's own error is of order h^2."""
    q, k, v, do = draw(1, 90, 90, 2, 1, 64, 30, gain=2.0)
    opts = dict(scale=0.125, causal=True, cap=cap)
    g = [t.to(DEV) for t in (q, k, v, do)]
    o, lse = rl.attention_forward(*g[:3], causal=True, softcap=cap)
    grads = rl.attention_backward(g[3], *g[:3], o, lse, causal=True, softcap=cap)
    base = [host(t) for t in (q, k, v)]
    bound = oa.run(*base, host(do), **opts)["bound"]
    loss = lambda x: float((oa.run(*x, **opts)["o"] * host(do)).sum())
    rng = np.random.default_rng(0)
    h = 1e-5
    for n, name in enumerate(("dq", "dk", "dv")):
        u = rng.standard_normal(base[n].shape)
        up = [x + h * u if i == n else x for i, x in enumerate(base)]
        down = [x - h * u if i == n else x for i, x in enumerate(base)]
        want = (loss(up) - loss(down)) / (2 * h)
        got = float((grads[n].double().cpu().numpy() * u).sum())
        assert abs(got - want) <= (bound[name] * np.abs(u)).sum() + 1e-4


# ---------------------------------------------------------------- one token

def check_token(B, n, hq, hk, d, lengths, cap=0.0, slopes=None, seed=0, fill=None):
    q, k, v, _ = draw(B, 1, n, hq, hk, d, seed, gain=3.0 if cap else 1.0)
    length = torch.tensor(lengths, dtype=torch.int32)
    rk, rv = k.clone(), v.clone()
    for b in range(B):
        if fill is not None:
            k[b, lengths[b]:] = fill
            v[b, lengths[b]:] = fill
    o = rl.attention_decode(q[:, 0].to(DEV), k.to(DEV), v.to(DEV), length.to(DEV), softcap=cap,
                            slopes=None if slopes is None else slopes.to(DEV))
    torch.cuda.synchronize()
    rl.device_status()
    for b in range(B):
        m = min(max(lengths[b], 0), n)
        if m == 0:
            assert (o[b] == 0).all()
            continue
        ref = oa.run(host(q[b:b + 1]), host(rk[b:b + 1, :m]), host(rv[b:b + 1, :m]),
                     scale=d ** -0.5, cap=cap, slopes=host(slopes))
        compare(dict(o=o[b:b + 1, None]), ref, ["o"])


@pytest.mark.parametrize("d", [8, 64, 80, 96, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (8, 2), (40, 8), (8, 8), (24, 1)])
def test_token_heads(hq, hk, d):
    check_token(3, 300, hq, hk, d, [300, 17, 256], seed=d + hq)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 4099])
def test_token_lengths(n):
    check_token(2, n, 8, 2, 128, [n, n - 1], seed=n)
    check_token(1, n, 4, 4, 64, [n], seed=n, cap=20.0)


def test_token_over_a_long_cache():
    check_token(1, 40001, 8, 2, 128, [40001], seed=3)
    check_token(2, 20000, 4, 1, 64, [19999, 3], seed=3, slopes=slopes_of(4))


def test_token_empty_negative_and_too_long_lengths():
    check_token(4, 200, 4, 2, 64, [0, -5, 1, 1000], seed=2)
    check_token(2, 0, 4, 2, 64, [0, 3], seed=2)


@pytest.mark.parametrize("cap,bias", [(15.0, False), (0.0, True), (15.0, True)])
def test_token_cap_and_bias(cap, bias):
    check_token(2, 777, 8, 2, 128, [777, 130], cap=cap, slopes=slopes_of(8) if bias else None)


def test_token_never_reads_past_the_length():
    check_token(3, 700, 8, 2, 128, [513, 1, 64], fill=float("nan"))
    check_token(3, 700, 8, 2, 64, [700, 0, 65], fill=float("inf"))


def test_token_cache_layouts():
    """[batch, heads, positions, dim] seen through a transpose, and a slice of one."""
    q, k, v, _ = draw(2, 1, 300, 4, 2, 64, 5)
    kk = k.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    vv = torch.cat((v, v), -1).to(DEV)[..., :64]
    n = torch.tensor([300, 100], dtype=torch.int32, device=DEV)
    a = rl.attention_decode(q[:, 0].to(DEV), kk, vv, n)
    b = rl.attention_decode(q[:, 0].to(DEV), k.to(DEV), v.to(DEV), n)
    assert torch.equal(a, b)


def test_token_repeats_bit_for_bit():
    q, k, v, _ = (t.to(DEV) for t in draw(2, 1, 9000, 8, 2, 128, 6))
    n = torch.tensor([9000, 5000], dtype=torch.int32, device=DEV)
    first = rl.attention_decode(q[:, 0], k, v, n)
    for _ in range(5):
        assert torch.equal(first, rl.attention_decode(q[:, 0], k, v, n))


def test_refuses_a_wrong_lse():
    q, k, v, _ = (t.to(DEV) for t in draw(2, 30, 30, 2, 1, 64, 1))
    good = torch.empty(2, 2, 30, device=DEV)
    rl.attention_forward(q, k, v, lse=good)
    for bad in (good[:, :1], good.half(), good.transpose(1, 2).contiguous(), good.cpu(),
                torch.empty(2, 2, 60, device=DEV)[:, :, ::2]):
        with pytest.raises(ValueError, match="lse"):
            rl.attention_forward(q, k, v, lse=bad)


def test_nothing_to_do():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)
    o, lse = rl.attention_forward(e(0, 5, 4, 64), e(0, 5, 2, 64), e(0, 5, 2, 64))
    assert o.shape == (0, 5, 4, 64)
    o, lse = rl.attention_forward(e(2, 0, 4, 64), e(2, 5, 2, 64), e(2, 5, 2, 64))
    dq, dk, dv = rl.attention_backward(e(2, 0, 4, 64), e(2, 0, 4, 64), e(2, 5, 2, 64),
                                       e(2, 5, 2, 64), o, lse)
    assert (dk == 0).all() and (dv == 0).all()
    assert rl.attention_decode(e(0, 4, 64), e(0, 9, 2, 64), e(0, 9, 2, 64),
                               torch.empty(0, dtype=torch.int32, device=DEV)).shape == (0, 4, 64)
