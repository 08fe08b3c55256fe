"""The root-mean-square norm, its gradients and its 8-bit output against the 64-bit
definition (needs a GB300).

Bounds.  U is half a step of the type (bf16 2^-8, fp32 2^-24), F = 2^-24.
h: the sum of two numbers in fp32 and, with dropout, a product by a factor off
   by F, then one rounding: U |h| + 3 F (|drop(x)| + |residual|).
rstd: sums of at most 32 + 10 positive terms a path (F each, halved by the root),
   a division and a root: 24 F; y adds two products and a rounding:
   (U + 28 F) |y|.  The norm is of the stored h, which the reference takes too.
codes: half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below the
   smallest normal number) and y's own 28 F.
dh: the mean has 42 terms a path, each of two products (50 F of the sum of
   magnitudes); d = r (g - hat c) + dh.
dw: a block adds its rows one after the other, then 8 lines of blocks: at most
   rows + 8 steps of F of the sum of magnitudes, and a rounding.
"""
import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import norm as on
from rank_linear_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: F}


def host(t):
    return t.detach().double().cpu().numpy().reshape(-1, t.shape[-1])


def make(rows, dim, dtype, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    return ((r(rows, dim) * scale).to(dtype), (r(rows, dim) * 2 * scale).to(dtype),
            (1 + 0.3 * r(dim)).to(dtype), r(rows, dim).to(dtype), r(rows, dim).to(dtype))


def check_forward(x, res, w, eps, out, p=0.0, seed=0, offset=0):
    y, h, rstd = out[:3]
    u = U[x.dtype]
    if res is not None or p:
        a = on.dropout(host(x), p, seed, offset)
        b = host(res) if res is not None else 0.0
        assert np.all(np.abs(host(h) - (a + b)) <= u * np.abs(a + b) + 3 * F * (np.abs(a) + np.abs(b)))
    else:
        assert h is x
    want, r = on.forward(host(h), host(w[None])[0], eps)
    assert np.all(np.abs(rstd.double().cpu().numpy().ravel() - r) <= 24 * F * r)
    assert np.all(np.abs(host(y) - want) <= (u + 28 * F) * np.abs(want) + 2.0 ** -133)
    if len(out) > 3:
        codes, scale = out[3:]
        s = scale.double().cpu().numpy().ravel()
        lo, hi = on.row_scale(want * (1 - 28 * F)), on.row_scale(want * (1 + 28 * F))
        assert np.all((s == lo) | (s == hi))
        got = host(codes.view(torch.float8_e4m3fn).float()) * s[:, None]
        assert np.all(np.abs(got - want) <= (2.0 ** -4 + 30 * F) * np.abs(want) + 2.0 ** -10 * s[:, None])


def check_backward(dy, h, w, rstd, dh, got, p=0.0, seed=0, offset=0):
    dx, dres, dw = got
    u = U[dy.dtype]
    y64, h64, w64 = host(dy), host(h), host(w[None])[0]
    r = rstd.double().cpu().numpy().ravel()
    d, dw64 = on.backward(y64, h64, w64, r, None if dh is None else host(dh))
    hat = h64 * r[:, None]
    g = np.abs(y64 * w64)
    tol = r[:, None] * (4 * F * g + 60 * F * np.abs(hat) * np.mean(g * np.abs(hat), -1, keepdims=True)) + \
        2 * F * np.abs(d) + (0 if dh is None else 2 * F * np.abs(host(dh)))
    assert np.all(np.abs(host(dres) - d) <= u * np.abs(d) + 1.01 * tol + 1e-38)
    if p:
        keep = 2.0 ** 32 / (2 ** 32 - round(p * 2 ** 32))
        want = on.dropout(d, p, seed, offset)
        assert np.all(np.abs(host(dx) - want) <= (u + 2 * F) * np.abs(want) + 1.01 * keep * tol * (want != 0) + 1e-38)
    else:
        assert dx is dres
    if dw is not None:
        terms = np.sum(np.abs(y64 * hat), 0)
        uw = U[dw.dtype]
        assert np.all(np.abs(host(dw[None])[0] - dw64) <= uw * np.abs(dw64) + (len(r) + 12) * F * terms + 1e-38)


DIMS = [1, 2, 7, 8, 31, 64, 100, 128, 136, 256, 264, 511, 512, 1000, 1024, 1032, 2001, 4096, 5120, 8192, 8200]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows", [1, 37, 700])
def test_forward_and_backward(rows, dim, dtype):
    x, res, w, dy, dh = make(rows, dim, dtype, seed=dim)
    residual, grad_in = (res, dh) if dim % 3 else (None, None)
    fp8 = rows != 37
    out = rl.rms_norm_forward(x, w, residual=residual, eps=1e-5, fp8=fp8)
    check_forward(x, residual, w, 1e-5, out)
    _, h, rstd = out[:3]
    got = rl.rms_norm_backward(dy, h, w, rstd, dh=grad_in)
    check_backward(dy, h, w, rstd, grad_in, got)
    again = rl.rms_norm_backward(dy, h, w, rstd, dh=grad_in)
    assert torch.equal(got[0], again[0]) and torch.equal(got[2], again[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(3, 32768), (5, 20001), (400, 16384)])
def test_the_widest(rows, dim, dtype):
    x, res, w, dy, dh = make(rows, dim, dtype, seed=7)
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-6, fp8=True, dropout=0.2, seed=3)
    check_forward(x, res, w, 1e-6, out, 0.2, 3)
    got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh, dropout=0.2, seed=3)
    check_backward(dy, out[1], w, out[2], dh, got, 0.2, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [5, 96, 777, 4096])
@pytest.mark.parametrize("residual", [True, False])
def test_dropout_of_the_branch(dim, residual, dtype):
    x, res, w, dy, dh = make(350, dim, dtype, seed=dim)
    res, dh = (res, dh) if residual else (None, None)
    drop = dict(dropout=0.3, seed=2 ** 63 + 11, offset=4)
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, **drop)
    check_forward(x, res, w, 1e-5, out, 0.3, 2 ** 63 + 11, 4)
    got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh, **drop)
    check_backward(dy, out[1], w, out[2], dh, got, 0.3, 2 ** 63 + 11, 4)


def test_fp32_weight_of_bf16_rows():
    x, res, w, dy, dh = make(65, 640, torch.bfloat16)
    w = w.float() + 1e-3
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, fp8=True)
    check_forward(x, res, w, 1e-5, out)
    got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh)
    assert got[2].dtype == torch.float32
    check_backward(dy, out[1], w, out[2], dh, got)
    assert rl.rms_norm_backward(dy, out[1], w, out[2], need_dweight=False)[2] is None


def test_strided_heads_and_odd_addresses():
    """The q heads of a fused q|k|v output, rows at odd addresses, a broadcast residual."""
    g = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn(50, 12, 80, generator=g, device=DEV).bfloat16()
    w = torch.rand(80, generator=g, device=DEV).bfloat16()
    q = qkv[:, 2:10]
    out = rl.rms_norm_forward(q, w, eps=1e-6)
    check_forward(q, None, w, 1e-6, out)
    dy = torch.randn(50, 8, 80, generator=g, device=DEV).bfloat16()
    dx = torch.zeros_like(qkv)
    got = rl.rms_norm_backward(dy, q, w, out[2], dx=dx[:, 2:10])
    check_backward(dy, q, w, out[2], None, (got[0], got[0], got[2]))
    assert torch.all(dx[:, :2] == 0) and torch.all(dx[:, 10:] == 0)
    flat = torch.randn(40 * 101 + 1, generator=g, device=DEV).bfloat16()
    x = flat[1:].view(40, 101)[:, :80]
    res = torch.randn(80, generator=g, device=DEV).bfloat16().expand(40, 80)
    check_forward(x, res, w, 1e-6, rl.rms_norm_forward(x, w, residual=res, eps=1e-6))
    with pytest.raises(ValueError):
        rl.rms_norm_forward(qkv.view(5, 10, 12, 80)[:, :7, :5], w)
    with pytest.raises(ValueError):
        rl.rms_norm_forward(qkv.transpose(1, 2), w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,heads,dim", [
    (400, 32, 128), (611, 20, 64), (350, 17, 128), (900, 129, 8), (333, 24, 256), (2048, 40, 32),
    (310, 6, 256)])
@pytest.mark.parametrize("strided", [False, True])
def test_heads_side_by_side(tokens, heads, dim, strided, dtype):
    """Rows narrow enough for a warp, taken `heads` at a time: with a residual, dropout,
    codes and every gradient."""
    g = torch.Generator(device=DEV).manual_seed(dim + heads)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)
    x, res, dy, dh = (r(tokens, heads + (3 if strided else 0), dim)[:, :heads] for _ in range(4))
    w = (1 + 0.3 * torch.randn(dim, generator=g, device=DEV)).to(dtype)
    out = rl.rms_norm_forward(x, w, eps=1e-5)
    check_forward(x, None, w, 1e-5, out)
    got = rl.rms_norm_backward(dy, x, w, out[2])
    check_backward(dy, x, w, out[2], None, got)
    drop = dict(dropout=0.3, seed=77, offset=1)
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, fp8=True, **drop)
    check_forward(x, res, w, 1e-5, out, 0.3, 77, 1)
    got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh, **drop)
    check_backward(dy, out[1], w, out[2], dh, got, 0.3, 77, 1)
    again = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh, **drop)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_heads_of_contiguous_rows():
    """The same of plain rows: [12800, 128] is taken 32 rows at a time, [12801, 128] is not."""
    for rows in (12800, 12801, 6400 * 3):
        x, res, w, dy, dh = make(rows, 128, torch.bfloat16, seed=rows)
        out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5)
        check_forward(x, res, w, 1e-5, out)
        a, b = x.clone(), res.clone()
        y, h, _ = rl.rms_norm_forward(a, w, residual=b, eps=1e-5, out=a, h_out=b)
        assert torch.equal(y, out[0]) and torch.equal(h, out[1])
        got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh)
        check_backward(dy, out[1], w, out[2], dh, got)


def test_in_place():
    x, res, w, dy, dh = make(33, 264, torch.bfloat16)
    y, h, rstd = rl.rms_norm_forward(x, w, residual=res)
    a, b = x.clone(), res.clone()
    y2, h2, _ = rl.rms_norm_forward(a, w, residual=b, out=a, h_out=b)
    assert y2 is a and h2 is b and torch.equal(a, y) and torch.equal(b, h)
    dx, _, dw = rl.rms_norm_backward(dy, h, w, rstd, dh=dh)
    e = dh.clone()
    dx2, _, dw2 = rl.rms_norm_backward(dy, h, w, rstd, dh=e, dx=e)
    assert dx2 is e and torch.equal(e, dx) and torch.equal(dw, dw2)
    with pytest.raises(ValueError):
        rl.rms_norm_forward(x, w, h_out=b)
    with pytest.raises(_lib.LoraError):
        rl.rms_norm_forward(x, w, residual=res, out=a, h_out=a)


def test_large_small_and_not_finite_rows():
    dim = 512
    x = torch.randn(6, dim, device=DEV)
    x[0] *= 1e30            # the squares leave fp32
    x[1] *= 1e-30           # eps decides
    x[2] = 0
    x[3, 5] = np.inf
    x[4, 7] = np.nan
    w = torch.ones(dim, device=DEV)
    y, _, rstd, codes, scale = rl.rms_norm_forward(x, w, eps=1e-6, fp8=True)
    want, r = on.forward(host(x[:3]), np.ones(dim), 1e-6)
    assert np.all(np.abs(host(y[:3]) - want) <= 40 * F * np.abs(want) + 1e-38)
    assert np.all(np.abs(rstd[:3].double().cpu().numpy() - r) <= 40 * F * r)
    assert torch.all(y[2] == 0) and torch.all(codes[2] == 0) and scale[2] == 1
    assert torch.isnan(y[3, 5]) and torch.all(y[3, :5] == 0)
    assert torch.isnan(y[4]).all() and torch.isfinite(y[5]).all()
    big = torch.full((2, 64), 3e38, device=DEV).bfloat16()
    y = rl.rms_norm_forward(big, torch.ones(64, device=DEV).bfloat16(), eps=0.0)[0]
    assert torch.all((y.float() - 1).abs() <= 2.0 ** -8)


def test_autograd_matches_the_functions_and_differences():
    x, res, w, dy, dh = make(20, 40, torch.float32)
    leaves = [t.clone().requires_grad_() for t in (x, w, res)]
    y, h = rl.rms_norm(leaves[0], leaves[1], residual=leaves[2], eps=1e-3, dropout=0.25, seed=5, offset=2)
    ((y * dy).sum() + (h * dh).sum()).backward()
    keep = torch.from_numpy(on.dropout(np.ones((20, 40)), 0.25, 5, 2)).to(DEV)
    ref = [t.double().requires_grad_() for t in (x, w, res)]
    h64 = ref[0] * keep + ref[2]
    y64 = h64 * (h64.square().mean(-1, keepdim=True) + 1e-3).rsqrt() * ref[1]
    ((y64 * dy.double()).sum() + (h64 * dh.double()).sum()).backward()
    for a, b in zip(leaves, ref):
        assert torch.allclose(a.grad.double(), b.grad, rtol=1e-5, atol=2e-5)
    # only one of the outputs used
    for pick in (0, 1):
        for t in leaves:
            t.grad = None
        rl.rms_norm(leaves[0], leaves[1], residual=leaves[2])[pick].sum().backward()
        assert all(torch.isfinite(t.grad).all() for t in leaves)
    assert torch.equal(leaves[0].grad, torch.ones_like(x)) and torch.all(leaves[1].grad == 0)
    # strides that the kernels do not take
    z = torch.randn(40, 20, device=DEV).t().requires_grad_()
    rl.rms_norm(z, leaves[1]).sum().backward()
    assert z.grad.shape == z.shape
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(rl.rms_norm(z, leaves[1]).sum(), z, create_graph=True)
        g.sum().backward()


def test_fp8_rows_feed_the_layer():
    """norm -> fp8 layer: the layer on the norm's codes, against it on its own, which
    quantises the rounded y: each within half a step of e4m3 of exact products."""
    g = torch.Generator(device=DEV).manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, res = r(300, 256).bfloat16(), r(300, 256).bfloat16()
    w = (1 + 0.1 * r(256)).bfloat16()
    W = rl.quantize_w_fp8((r(320, 256) / 16).bfloat16())
    A, B = (r(16, 256) / 16).bfloat16().requires_grad_(), (r(320, 16) * 0.1).bfloat16().requires_grad_()
    y, h, codes, scale = rl.rms_norm(x, w, residual=res, fp8=True)
    got = rl.lora_linear_fp8(y, W, A, B, 32.0, rows=(codes, scale))
    # the same codes through the layer's own quantiser's format
    q = (codes.view(torch.float8_e4m3fn).float() * scale[:, None]).double()
    Wd = W.Wq.view(torch.float8_e4m3fn).float().double() * W.w_scale.double()
    want = q @ Wd.T + 2.0 * (y.double() @ A.double().T) @ B.double().T
    assert float((got.double() - want).detach().abs().max() / want.detach().abs().max()) <= 1e-2
    got.sum().backward()
    ga = A.grad.clone()
    A.grad = B.grad = None
    rl.lora_linear_fp8(y, W, A, B, 32.0).sum().backward()
    assert torch.equal(A.grad, ga)
    plain, _ = rl.fp8_forward(y, W, A.detach(), B.detach(), 32.0, rows=rl.quantize_rows_fp8(y))
    own, _ = rl.fp8_forward(y, W, A.detach(), B.detach(), 32.0)
    assert torch.equal(plain, own)
    with pytest.raises(ValueError):
        rl.fp8_forward(y, W, A.detach(), B.detach(), 32.0, rows=(codes[:1], scale[:1]))
    rl.device_status()


def test_no_rows():
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, device=DEV)
    y, h, rstd = rl.rms_norm_forward(x, w, residual=x)
    dx, _, dw = rl.rms_norm_backward(x, h, w, rstd, dh=x)
    assert y.shape == dx.shape == (0, 64) and torch.all(dw == 0)
    with pytest.raises(TypeError):
        rl.rms_norm_forward(x, w.double())
    with pytest.raises(ValueError):
        rl.rms_norm_forward(x, w[:32])


def test_graph_replay_and_streams():
    x, res, w, dy, dh = make(64, 512, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, h, rstd = rl.rms_norm_forward(x, w, residual=res)
        rl.rms_norm_backward(dy, h, w, rstd, dh=dh)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, rstd = rl.rms_norm_forward(x, w, residual=res)
        dx, _, dw = rl.rms_norm_backward(dy, h, w, rstd, dh=dh)
    x.mul_(1.5)
    graph.replay()
    y2, h2, rstd2 = rl.rms_norm_forward(x, w, residual=res)
    want = rl.rms_norm_backward(dy, h2, w, rstd2, dh=dh)
    assert torch.equal(y, y2) and torch.equal(dx, want[0]) and torch.equal(dw, want[2])
    side.wait_stream(torch.cuda.current_stream())
    y3, h3, rstd3 = rl.rms_norm_forward(x, w, residual=res, stream=side)
    got = rl.rms_norm_backward(dy, h3, w, rstd3, dh=dh, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y3, y2) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [513, 1001, 1030, 2001, 2046, 4095, 4097, 5121, 8178, 8185])
@pytest.mark.parametrize("lead,pad", [(0, 0), (3, 1), (1, 7)])
def test_rows_off_the_16_byte_boundaries(dim, lead, pad, dtype):
    """More rows than blocks, which begin anywhere: every tensor alike, then one otherwise."""
    rows = 1000 if dim < 3000 else 500
    g = torch.Generator(device=DEV).manual_seed(dim + lead)
    step = dim + pad

    def room(off):
        t = torch.full((rows * step + off + 1,), 7.0, dtype=dtype, device=DEV)
        return t, t[off:].as_strided((rows, dim), (step, 1))
    rand = lambda off: room(off)[1].copy_(torch.randn(rows, dim, generator=g, device=DEV))
    x, res, dy, dh = (rand(lead) for _ in range(4))
    w = (1 + 0.3 * torch.randn(dim, generator=g, device=DEV)).to(dtype)
    for off in (lead, lead + 1):
        (ty, y), (th, h), (td, d) = (room(o) for o in (off, lead, lead))
        out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, out=y, h_out=h, fp8=pad == 0)
        check_forward(x, res, w, 1e-5, out)
        got = rl.rms_norm_backward(dy, h, w, out[2], dh=dh, dx=d)
        check_backward(dy, h, w, out[2], dh, got)
        again = rl.rms_norm_backward(dy, h, w, out[2], dh=dh, dx=d)
        assert torch.equal(got[2], again[2])
        for flat, part in ((ty, y), (th, h), (td, d)):
            part.fill_(7.0)
            assert torch.all(flat == 7.0)  # nothing beside the rows was written
    out = rl.rms_norm_forward(x, w, eps=1e-5)
    check_forward(x, None, w, 1e-5, out)
    check_backward(dy, x, w, out[2], None, rl.rms_norm_backward(dy, x, w, out[2]))
    # in place the bits of the same layout elsewhere (another has its sums in another order)
    want = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, out=room(lead)[1], h_out=room(lead)[1])
    y, h, rstd = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, out=x, h_out=res)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and torch.equal(rstd, want[2])
    rl.device_status()


def test_not_finite_neighbours_of_rows_off_the_boundaries():
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(901, 1003, device=DEV).to(dtype)
        w = torch.ones(1003, device=DEV, dtype=dtype)
        want = rl.rms_norm_forward(x, w)
        x[1::2] = float("nan")
        got = rl.rms_norm_forward(x, w)
        assert torch.equal(got[0][::2], want[0][::2]) and torch.equal(got[2][::2], want[2][::2])
        dx, _, _ = rl.rms_norm_backward(x, x, w, got[2])
        assert torch.isfinite(dx[::2]).all() and torch.isnan(dx[1::2]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,lead,w_lead", [(2048, 3, 0), (2048, 0, 1), (1056, 1, 3), (4096, 5, 5)])
def test_whole_vectors_at_odd_addresses(dim, lead, w_lead, dtype):
    """Widths of whole vectors whose rows, or whose weight alone, begin off 16 bytes."""
    g = torch.Generator(device=DEV).manual_seed(dim + lead)
    make_rows = lambda: torch.randn(600 * dim + lead, generator=g, device=DEV).to(dtype)[lead:].view(600, dim)
    x, res, dy, dh, y, h, dx = (make_rows() for _ in range(7))
    w = torch.randn(dim + w_lead, generator=g, device=DEV).to(dtype)[w_lead:]
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, out=y, h_out=h)
    check_forward(x, res, w, 1e-5, out)
    got = rl.rms_norm_backward(dy, h, w, out[2], dh=dh, dx=dx)
    check_backward(dy, h, w, out[2], dh, got)
    rl.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [8, 40, 48, 56, 72, 80, 96, 104, 160, 168, 192, 232, 248, 520, 640, 768, 776])
def test_narrow_rows_of_whole_vectors(dim, dtype):
    """Widths whose vectors fill the threads' three or four, and do not; plain rows and heads."""
    for shape in ((3001,), (400, 24), (512, 9)):
        g = torch.Generator(device=DEV).manual_seed(dim)
        r = lambda: torch.randn(*shape, dim, generator=g, device=DEV).to(dtype)
        x, res, dy, dh = r(), r(), r(), r()
        w = (1 + 0.3 * torch.randn(dim, generator=g, device=DEV)).to(dtype)
        out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5)
        check_forward(x, res, w, 1e-5, out)
        got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh)
        check_backward(dy, out[1], w, out[2], dh, got)
    rl.device_status()


# One shape a kernel: few rows, narrow rows, heads, the ring on and off the boundaries, element by
# element, and rows too wide for the ring.
FORMS = [(7, 512), (3001, 96), (12800, 128), (900, 4096), (1000, 1001), (700, 300), (8, 20001), (310, 8200)]


def scaled_rows(rows, dim, dtype, scales, seed):
    """(x, dy, w, factor of each row): rows on the scales in turn, and dy partly along them, of size 1e6
    (no gradient is as small as the checks' 1e-38)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    unit = r(rows, dim)
    s = torch.tensor(scales, device=DEV).repeat(rows // len(scales) + 1)[:rows, None]
    return ((unit * s).to(dtype), ((r(rows, dim) + unit) * 1e6).to(dtype), (1 + 0.3 * r(dim)).to(dtype), s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", FORMS)
def test_gradients_of_large_rows(rows, dim, dtype):
    """Rows whose squares, or the square of whose rstd, leave fp32, beside ordinary ones: every
    gradient, within the bounds of ordinary rows."""
    x, dy, w, s = scaled_rows(rows, dim, dtype, [1.0, 1e18, 1e21, 1e22, 1e25, 1e30, 1e36], dim)
    out = rl.rms_norm_forward(x, w, eps=1e-6)
    check_forward(x, None, w, 1e-6, out)
    check_backward(dy, x, w, out[2], None, rl.rms_norm_backward(dy, x, w, out[2]))
    # what reaches h otherwise, as small as the rest
    dh = (dy.float() / s).to(dtype)
    check_backward(dy, x, w, out[2], dh, rl.rms_norm_backward(dy, x, w, out[2], dh=dh))
    rl.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(3, 8192), (400, 8192), (700, 6001), (2, 32768), (310, 16384)])
def test_wide_rows_of_the_largest_numbers(rows, dim, dtype):
    """Rows whose squares leave fp32 although each is scaled down by 2^-70.  rstd is below 2^-126 and
    so a multiple of 2^-149: 2^-22 of it at most, which y has as well."""
    g = torch.Generator(device=DEV).manual_seed(dim)
    sign = torch.randint(0, 2, (rows, dim), generator=g, device=DEV) * 2 - 1
    x = (sign * 3e38).to(dtype)
    x[1:, ::2] = sign[1:, ::2].to(dtype)  # (beside it a row of which half the elements count)
    w = (1 + 0.3 * torch.randn(dim, generator=g, device=DEV)).to(dtype)
    y, _, rstd = rl.rms_norm_forward(x, w, eps=1e-6)
    want, r = on.forward(host(x), host(w[None])[0], 1e-6)
    assert np.all(np.abs(rstd.double().cpu().numpy() - r) <= (24 * F + 2.0 ** -22) * r)
    assert np.all(np.abs(host(y) - want) <= (U[dtype] + 28 * F + 2.0 ** -22) * np.abs(want) + 2.0 ** -133)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", FORMS)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -116])
def test_small_rows_where_eps_is_small(rows, dim, eps, dtype):
    """Rows whose squares have lost their bits, or are 0, beside ordinary ones, with an eps that does
    not hide it: outputs and every gradient, within the bounds of ordinary rows."""
    x, dy, w, s = scaled_rows(rows, dim, dtype, [1.0, 1e-14, 1e-18, 1e-20, 1e-23, 1e-30, 1e-36], dim)
    dy = dy * 1e-6  # (gradients are as large as rstd: 1e36)
    out = rl.rms_norm_forward(x, w, eps=eps)
    check_forward(x, None, w, eps, out)
    check_backward(dy, x, w, out[2], None, rl.rms_norm_backward(dy, x, w, out[2]))
    dh = (dy.float() / s).to(dtype)
    check_backward(dy, x, w, out[2], dh, rl.rms_norm_backward(dy, x, w, out[2], dh=dh))
    rl.device_status()


def dw_of_many(dy, h, rstd, dw):
    """dw against 64 bits: a block adds its rows one after the other, at most as many as come on one of
    an SM's blocks each, then its groups of threads, and the join an eighth of at most 12 blocks' lines an
    SM, and eight."""
    rows = h.shape[0]
    terms = dy.double() * h.double() * rstd.double()[..., None]
    lead = tuple(range(h.dim() - 1))
    steps = rows / 152 + 12 * 152 / 8 + 64
    bound = U[dw.dtype] * terms.sum(lead).abs() + steps * F * terms.abs().sum(lead)
    assert torch.all((dw.double() - terms.sum(lead)).abs() <= bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,lead", [
    ((4500, 4096), 0), ((3000, 4097), 1), ((17000, 1001), 3), ((17000, 513), 0), ((1500, 8185), 0), ((1500, 8192), 0),
    ((3000, 32, 128), 0), ((4500, 40, 96), 0), ((9000, 24, 96), 0), ((11000, 1030), 1)])
def test_every_stage_of_the_ring_many_times(shape, lead, dtype):
    """So many rows (of heads side by side: tokens) that each block fills every stage of its ring more
    than twice.  Parts of them, which fill none twice, have the same bits: the rows lie alike in both."""
    g = torch.Generator(device=DEV).manual_seed(shape[0])
    n, heads, dim = shape[0], shape[1:-1], shape[-1]
    room = (n, *(k + 2 for k in heads), dim)  # (two heads more, so that tokens are apart)
    size = torch.Size(room).numel()

    def rand():
        t = torch.randn(size + lead, generator=g, device=DEV).to(dtype)[lead:].view(room)
        return t[:, :heads[0]] if heads else t
    x, res, dy, dh, y, h, dx = (rand() for _ in range(7))
    w = (1 + 0.3 * torch.randn(shape[-1], generator=g, device=DEV)).to(dtype)
    _, _, rstd = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, out=y, h_out=h)
    _, _, dw = rl.rms_norm_backward(dy, h, w, rstd, dh=dh, dx=dx)
    for at in range(0, n, 8 * (n // 72)):
        part = slice(at, min(at + 400, n))
        if part.stop - at < 310:
            part = slice(n - 8 * (310 // 8 + 1) - n % 8, n)  # (the last rows, from a multiple of eight on)
        out = rl.rms_norm_forward(x[part], w, residual=res[part], eps=1e-5, out=rand()[part], h_out=rand()[part])
        got = rl.rms_norm_backward(dy[part], h[part], w, rstd[part], dh=dh[part], dx=rand()[part], need_dweight=False)
        assert torch.equal(out[0], y[part]) and torch.equal(out[1], h[part]) and torch.equal(out[2], rstd[part])
        assert torch.equal(got[0], dx[part])
    dw_of_many(dy, h, rstd, dw)
    rl.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(12000, 1001), (3000, 4097), (4500, 4096), (1500, 8191)])
def test_dropped_out_rows_through_every_stage(rows, dim, dtype):
    """The same with dropout, whose masks go by the row, on the boundaries and element by element."""
    x, res, w, dy, dh = make(rows, dim, dtype, seed=rows)
    drop = dict(dropout=0.25, seed=12, offset=3)
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, **drop)
    check_forward(x, res, w, 1e-5, out, 0.25, 12, 3)
    got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh, **drop)
    check_backward(dy, out[1], w, out[2], dh, got, 0.25, 12, 3)
    dw_of_many(dy, out[1], out[2], got[2])
    rl.device_status()


@pytest.mark.parametrize("rows,dim", FORMS + [(4500, 4096), (2000, 4097), (400, 8192)])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_fp32_weights_in_every_form(rows, dim, p):
    """bf16 rows under weights that bf16 does not hold, with everything else that a call may have."""
    x, res, w, dy, dh = make(rows, dim, torch.bfloat16, seed=rows + dim)
    w = w.float() * (1 + 2.0 ** -12)
    drop = dict(dropout=p, seed=21, offset=6) if p else {}
    out = rl.rms_norm_forward(x, w, residual=res, eps=1e-5, fp8=True, **drop)
    check_forward(x, res, w, 1e-5, out, p, 21, 6)
    got = rl.rms_norm_backward(dy, out[1], w, out[2], dh=dh, **drop)
    assert got[2].dtype == torch.float32
    check_backward(dy, out[1], w, out[2], dh, got, p, 21, 6)
    rl.device_status()
