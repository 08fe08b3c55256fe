"""Attention where it can go wrong beyond the usual sizes and values: waits between
the warps of a block, extreme caps, few visible keys among many, tensors that the
kernels cannot take as they are (needs a GB300).

The reference and its bounds are those of test_gpu_attention.py.
"""
import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import attention as oa
from test_gpu_attention import DEV, check, draw, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_key_gradients_over_every_number_of_steps(d):
    """One to many query tiles for a block of dk and dv, again and again: no wait
    runs out and every run gives the same bits."""
    for sq in (100, 200, 300, 400, 520, 1500):
        q, k, v, do = (t.to(DEV) for t in draw(1, sq, 130, 2, 1, d, sq))
        o, lse = rl.attention_forward(q, k, v)
        first = rl.attention_backward(do, q, k, v, o, lse)
        for _ in range(30):
            again = rl.attention_backward(do, q, k, v, o, lse)
        torch.cuda.synchronize()
        rl.device_status()
        for a, b in zip(first, again):
            assert torch.equal(a, b)
    check(*draw(1, 1100, 260, 4, 1, d, 7))


def expanded(x, d):
    """x and its views with a broadcast head, a broadcast token, a broadcast batch
    entry, a strided head, an odd address; each with the values it stands for."""
    b, n, h, _ = x.shape
    wide = torch.randn(b, n, h, 2 * d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    odd = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
    odd.copy_(x)
    return [x[:, :, :1].expand(b, n, h, d), x[:, :1].expand(b, n, h, d), x[:1].expand(b, n, h, d),
            wide[..., ::2], odd, x[..., :1].expand(b, n, h, d), x.transpose(1, 2).contiguous().transpose(1, 2)]


@pytest.mark.parametrize("which", range(4))
def test_views_that_autograd_copies(which):
    """attention() of q, k, v and an output gradient that the kernels do not take as
    they are: the bits of their contiguous copies."""
    d = 64
    x = [t.to(DEV) for t in draw(2, 150, 150, 4, 4, d, 3)]
    for view in expanded(x[which], d):
        t = list(x)
        t[which] = view
        leaf = [y.detach().requires_grad_() for y in t[:3]]
        o = rl.attention(*leaf, causal=True)
        o.backward(t[3])
        plain = [y.clone(memory_format=torch.contiguous_format) for y in t]
        o1, lse = rl.attention_forward(*plain[:3], causal=True)
        want = rl.attention_backward(plain[3], *plain[:3], o1, lse, causal=True)
        assert torch.equal(o, o1)
        for a, b in zip(leaf, want):
            assert torch.equal(a.grad, b)
    rl.device_status()


def test_broadcast_tensors_are_refused_or_read():
    q, k, v, do = (t.to(DEV) for t in draw(2, 60, 60, 4, 2, 64, 3))
    many = k[:, :, :1].expand(2, 60, 2, 64)
    with pytest.raises(rl._lib.LoraError, match="broadcast"):
        rl.attention_forward(q, many, v)
    n = torch.tensor([60, 17], dtype=torch.int32, device=DEV)
    one = rl.attention_decode(q[:, 0], k[:1].expand(2, 60, 2, 64), many, n)  # one prompt's cache for both
    two = rl.attention_decode(q[:, 0], k[:1].repeat(2, 1, 1, 1), many.contiguous(), n)
    assert torch.equal(one, two)


def whole_numbers(B, sq, sk, hq, hk, d, seed):
    """q and k of -1, 0 and 1: every score is exact in fp32, many are 0."""
    q, k, v, do = draw(B, sq, sk, hq, hk, d, seed)
    g = torch.Generator().manual_seed(seed)
    w = lambda t: torch.randint(-1, 2, t.shape, generator=g).bfloat16()
    return w(q), w(k), v, do


@pytest.mark.parametrize("cap", [1e-40, 1e-30, 1e-20, 1e-10, 1e-6, 1e-5, 2e-5, 1e-4, 1e-3])
@pytest.mark.parametrize("d", [64, 128])
def test_small_caps(cap, d):
    """Scores of 0, whose slope is 1, beside scores far beyond the cap; rows past the
    end in the last tile."""
    check(*whole_numbers(1, 190, 190, 4, 2, d, 3), causal=True, cap=cap)
    check(*whole_numbers(2, 50, 210, 2, 2, d, 4), cap=cap, scale=1.0)
    check(*whole_numbers(1, 150, 150, 2, 1, d, 5), causal=True, cap=cap,
          slopes=torch.tensor([0.25, 0.0625]))


@pytest.mark.parametrize("cap", [1.0, 50.0, 1e3, 1e4, 1e5, 1e7, 1e15, 1e25, 1e37])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_below_at_and_beyond_any_cap(cap, d):
    """Each query sees one key, its own document's: lse is the score, from 1/1000 of the
    cap to 10 times it within one warp.  q and k are positive: a score is off by 2^-17
    of itself (128 roundings of 2^-24), tanh by less than 2^-18, the unit of lse by 2^-22."""
    n = 256
    q, k, v, _ = draw(1, n, n, 2, 1, d, 11)
    q, k = q.abs(), k.abs()
    far = torch.logspace(-3, 1, n)[torch.randperm(n, generator=torch.Generator().manual_seed(2))]
    q = (q * far[None, :, None, None]).bfloat16()
    scale = float(np.float32(cap / (0.64 * d)))
    docs = torch.arange(n, dtype=torch.int32)[None]
    _, lse = rl.attention_forward(q.to(DEV), k.to(DEV), v.to(DEV), softcap=cap, scale=scale,
                                  documents=docs.to(DEV))
    z = scale * np.einsum("ihd,id->hi", q[0].double().numpy(), k[0, :, 0].double().numpy())
    capped = float(np.float32(cap))
    want = capped * np.tanh(z / capped)
    got = lse[0].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -16 * want)


@pytest.mark.parametrize("cap", [30.0, 1e4, 1e6])
@pytest.mark.parametrize("d", [64, 128])
def test_what_padding_holds_leaves_scores_below_a_large_cap_alone(cap, d):
    docs = torch.zeros(1, 300, dtype=torch.int32)
    docs[0, ::31] = -1
    q, k, v, do = draw(1, 300, 300, 2, 1, d, 8)
    for t in (q, k):
        t[docs < 0] = 1e15
    check(q, k, v, do, causal=True, cap=cap, docs=docs)
    check(q, k, v, do, cap=cap, docs=docs, slopes=torch.tensor([0.25, 0.0625]))


@pytest.mark.parametrize("cap", [1e-30, 1e-5, 1.0, 1e2, 1e3, 1e4, 1e5, 1e6, 1e15, 1e30])
@pytest.mark.parametrize("n", [2, 5, 700])
@pytest.mark.parametrize("d", [64, 128])
def test_token_with_any_cap(n, cap, d):
    """One new token's output: rounded once (U), from weights good to F in scores and
    2^-16 in their two bf16 parts; pv is what the weights' error goes through."""
    B, hq, hk = 2, 8, 2
    q, k, v, _ = (whole_numbers if cap < 1e-3 else draw)(B, 1, n, hq, hk, d, n + d)
    length = torch.full((B,), n, dtype=torch.int32)
    o = rl.attention_decode(q[:, 0].to(DEV), k.to(DEV), v.to(DEV), length.to(DEV), softcap=cap)
    ref = oa.run(host(q), host(k), host(v), scale=d ** -0.5, cap=cap)
    pv = ref["bound"]["o"][:, 0] / (2 * oa.U + oa.F)
    err = np.abs(o.double().cpu().numpy() - ref["o"][:, 0])
    assert np.all(err <= (oa.U + 2 * oa.F) * pv + 1e-30), (err / (pv + 1e-30)).max()


def test_token_beyond_the_cap_and_below_it():
    """Heads far beyond a large cap beside heads far below it in one warp."""
    q, k, v, _ = draw(1, 1, 40, 8, 1, 64, 5)
    q[:, :, 1::2] *= 1e7
    o = rl.attention_decode(q[:, 0].to(DEV), k.to(DEV), v.to(DEV),
                            torch.tensor([40], dtype=torch.int32, device=DEV), softcap=1e5)
    ref = oa.run(host(q), host(k), host(v), scale=0.125, cap=1e5)
    pv = ref["bound"]["o"][:, 0] / (2 * oa.U + oa.F)
    err = np.abs(o.double().cpu().numpy() - ref["o"][:, 0])[:, ::2]
    assert np.all(err <= (oa.U + 2 * oa.F) * pv[:, ::2])


def check_rows_of_one_tile(q, k, v, do, *, causal=False, cap=0.0, slopes=None, prefix=None, docs=None):
    """dq and dk with the bound of test_gpu_attention.few_keys for every query whose
    keys lie in one tile of 128, however many keys there are, and the reference's
    general bound for the others; how many such queries there were."""
    dev = lambda t: None if t is None else t.to(DEV)
    opts = dict(causal=causal, softcap=cap, slopes=dev(slopes), documents=dev(docs), prefix=dev(prefix))
    g = [dev(t) for t in (q, k, v, do)]
    o, lse = rl.attention_forward(*g[:3], **opts)
    got = dict(zip(("dq", "dk", "dv"), rl.attention_backward(g[3], *g[:3], o, lse, **opts)))
    torch.cuda.synchronize()
    rl.device_status()
    (B, sq, hq, d), (sk, hk) = q.shape, k.shape[1:3]
    scale, (q, k, v, do) = d ** -0.5, map(host, (q, k, v, do))
    G, M = 2.0 ** -12, 2.0 ** -16
    rows = 0
    for b in range(B):
        kd = None if docs is None else docs[b].numpy()
        see = oa.visible(sq, sk, causal, 0 if prefix is None else int(prefix[b]),
                         None if kd is None else kd[sk - sq:], kd)
        tiles = sum(see[:, t:t + 128].any(1).astype(int) for t in range(0, sk, 128))
        one = (tiles <= 1)[:, None]
        rows += int((tiles == 1).sum())
        for n in range(hk):
            dk, dkb = 0.0, 1e-30
            for h in range(n * (hq // hk), (n + 1) * (hq // hk)):
                p, sl, oo, _, qkv = oa.head(q[b, :, h], k[b, :, n], v[b, :, n], scale=scale, see=see, cap=cap,
                                            slope=0.0 if slopes is None else float(slopes[h]))
                grad = oa.head_backward(do[b, :, h], p, sl, oo, qkv, scale=scale, see=see)
                e, vv = np.abs(grad[4]), np.abs(qkv[2])
                dp, size, pv = np.abs(grad[4] @ qkv[2].T), e @ vv.T, p @ vv
                few = p * sl * (G * (dp + (p * dp).sum(1, keepdims=True))
                                + M * (size + (p * size).sum(1, keepdims=True)))
                many = p * sl * ((e * (2 * oa.U + oa.F) * pv).sum(1, keepdims=True)
                                 + oa.F * (size + (e * pv).sum(1, keepdims=True)))
                dz = np.where(one, 2 * oa.U * np.abs(grad[3]) + few,
                              (2 * oa.U + 2 * oa.F) * np.abs(grad[3]) + many)
                err = np.abs(got["dq"][b, :, h].double().cpu().numpy() - grad[0])
                bound = scale * dz @ np.abs(qkv[1]) + 1e-30
                assert np.all(err <= bound), ("dq", b, h, np.argwhere(err > bound)[:4].tolist(), (err / bound).max())
                dk, dkb = dk + grad[1], dkb + scale * dz.T @ np.abs(qkv[0])
            err = np.abs(got["dk"][b, :, n].double().cpu().numpy() - dk)
            assert np.all(err <= dkb), ("dk", b, n, (err / dkb).max())
    return rows


def uneven(B, sq, sk, hq, hk, d, seed):
    """Some keys draw most of their queries' weight, or none."""
    q, k, v, do = draw(B, sq, sk, hq, hk, d, seed)
    k[:, ::3] *= 3
    return q, k, v, do


@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, False), (0.0, True), (30.0, True)])
@pytest.mark.parametrize("sq,sk,d", [(129, 129, 128), (300, 300, 64), (520, 520, 128), (200, 260, 128),
                                     (260, 200, 64), (500, 129, 128)])
def test_first_rows_of_long_sequences(sq, sk, d, cap, bias):
    """The first queries of a causal mask see few keys, of however many there are."""
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625]) if bias else None
    assert check_rows_of_one_tile(*uneven(2, sq, sk, 4, 2, d, sq + sk), causal=True, cap=cap, slopes=slopes) > 0


def test_first_rows_with_a_prefix():
    x = uneven(2, 400, 400, 4, 2, 64, 6)
    assert check_rows_of_one_tile(*x, causal=True, prefix=torch.tensor([3, 100], dtype=torch.int32)) > 0
    x = uneven(2, 400, 250, 4, 2, 64, 7)
    assert check_rows_of_one_tile(*x, causal=True, prefix=torch.tensor([5, 200], dtype=torch.int32)) > 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("d", [64, 128])
def test_short_documents_among_many_keys(d, cap, causal):
    """Documents of 1 to 8 tokens, and longer ones between them; a document that a
    tile's edge cuts shares its tiles with whole ones."""
    g = torch.Generator().manual_seed(d)
    sizes = torch.randint(1, 9, (200,), generator=g).tolist()
    sizes[20], sizes[50], sizes[51] = 130, 100, 37
    row = sum(([i] * n for i, n in enumerate(sizes)), [])[:680]
    docs = torch.tensor([row + [-1] * 20, [-1] * 5 + row + [-1] * 15], dtype=torch.int32)
    rows = check_rows_of_one_tile(*uneven(2, 700, 700, 4, 2, d, 9), causal=causal, cap=cap, docs=docs)
    # of each row's 680 tokens the longer documents have 267, tiles' edges cut 5 others at most
    assert rows >= 2 * (680 - 267 - 5 * 8)
    # the last queries only
    q, k, v, do = uneven(2, 150, 700, 4, 2, d, 10)
    assert check_rows_of_one_tile(q, k, v, do, causal=causal, cap=cap, docs=docs) > 100


@pytest.mark.parametrize("sq,sk,kw", [
    (1500, 1500, {}), (1500, 1437, {}), (1437, 1500, {}), (1500, 1244, {}), (1500, 100, {}), (100, 1500, {}),
    (1500, 1437, dict(prefix=torch.tensor([90], dtype=torch.int32))),
    (1500, 1500, dict(prefix=torch.tensor([90], dtype=torch.int32))),
    (1500, 1500, dict(documents=(torch.arange(1500, dtype=torch.int32) // 7)[None]))])
def test_gradients_of_few_keys_repeat_bit_for_bit(sq, sk, kw):
    """dk and dv take delta that dq leaves: always the same one."""
    kw = {n: t.to(DEV) for n, t in kw.items()}
    g = [t.to(DEV) for t in uneven(1, sq, sk, 32, 2, 128, 3)]
    o, lse = rl.attention_forward(*g[:3], causal=True, **kw)
    first = rl.attention_backward(g[3], *g[:3], o, lse, causal=True, **kw)
    for _ in range(20):
        again = rl.attention_backward(g[3], *g[:3], o, lse, causal=True, **kw)
        for a, b in zip(first, again):
            assert torch.equal(a, b)
    rl.device_status()


def test_options_given_as_tensors_are_read_at_each_call():
    q, k, v, do = (t.to(DEV) for t in draw(1, 70, 70, 2, 1, 64, 4))
    scale, cap, causal = torch.tensor(0.1), torch.tensor(5.0), torch.tensor(False)
    n = torch.tensor([70], dtype=torch.int32, device=DEV)

    def both(scale, cap, causal):
        o, lse = rl.attention_forward(q, k, v, scale=scale, softcap=cap, causal=causal)
        grads = rl.attention_backward(do, q, k, v, o, lse, scale=scale, softcap=cap, causal=causal)
        return (o, lse) + grads + (rl.attention_decode(q[:, 0], k, v, n, scale=scale, softcap=cap),)

    for s, c, m in ((0.1, 5.0, False), (0.2, 5.0, False), (0.2, 9.0, False), (0.2, 9.0, True)):
        scale.fill_(s), cap.fill_(c), causal.fill_(m)
        for a, b in zip(both(scale, cap, causal), both(scale.item(), cap.item(), causal.item())):
            assert torch.equal(a, b), (s, c, m)
    # and the backward of attention() is that of its forward
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    o = rl.attention(*x, scale=scale, softcap=cap)
    was = scale.item()
    scale.fill_(0.7)
    o.backward(do)
    y = [t.clone().requires_grad_() for t in (q, k, v)]
    rl.attention(*y, scale=was, softcap=9.0).backward(do)
    for a, b in zip(x, y):
        assert torch.equal(a.grad, b.grad)
