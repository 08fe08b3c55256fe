"""The large-vocabulary loss and its gradient against the 64-bit oracle, within the
bounds that it derives (needs a GB300)."""
import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import head_loss as ol

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(rows, dim, vocab, seed=0, scale=1.0, ignored=0.3):
    g = torch.Generator(device=DEV).manual_seed(seed + rows + dim + vocab)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, w = (r(rows, dim) * scale).bfloat16(), (r(vocab, dim) * 2 * dim ** -0.5).bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    t[torch.rand(rows, generator=g, device=DEV) < ignored] = -100
    return x, w, t, torch.rand(rows, generator=g, device=DEV)


def host(t):
    return t.detach().double().cpu().numpy()


def check(got, x, w, t, weights=None, cap=0.0, mean=True):
    loss, losses, dx = got
    want = ol.run(host(x), host(w), t.cpu().numpy(), None if weights is None else host(weights), cap, mean,
                  dx is not None)
    assert np.all(np.abs(host(losses) - want["losses"]) <= want["e_losses"])
    assert abs(float(loss) - want["loss"]) <= want["e_loss"] + 2 * ol.F * abs(want["loss"])
    if dx is not None:
        assert np.all(np.abs(host(dx) - want["dx"]) <= want["e_dx"])
        assert torch.all(dx[t < 0] == 0)
    rl.device_status()


SIZES = [(1, 8, 1), (1, 64, 2), (3, 8, 7), (5, 72, 511), (31, 24, 640), (257, 128, 512), (300, 1000, 513),
         (256, 64, 1025), (129, 4096, 700), (513, 520, 4097), (700, 256, 33001)]


@pytest.mark.parametrize("rows,dim,vocab", SIZES)
@pytest.mark.parametrize("gradient", [False, True])
def test_sizes(rows, dim, vocab, gradient):
    x, w, t, _ = make(rows, dim, vocab)
    got = rl.cross_entropy_forward(x, w, t, gradient=gradient)
    check(got, x, w, t)
    again = rl.cross_entropy_forward(x, w, t, gradient=gradient)
    for a, b in zip(got, again):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("cap", [0.01, 0.5, 5.0, 30.0, 1e4])
@pytest.mark.parametrize("mean", [True, False])
def test_cap_and_weights(cap, mean):
    x, w, t, weights = make(200, 264, 1500, scale=3.0)
    got = rl.cross_entropy_forward(x, w, t.int(), weights=weights, softcap=cap, gradient=True,
                                   reduction="mean" if mean else "sum")
    check(got, x, w, t, weights, cap, mean)


@pytest.mark.parametrize("cap", [0.0, 500.0])
@pytest.mark.parametrize("scale", [8.0, 60.0, 500.0])
def test_certain_and_hopeless_targets(scale, cap):
    """Logits hundreds apart: exponentials relative to a hopeless target leave fp32 and
    are kept on other scales; half the targets are the likeliest words."""
    x, w, t, _ = make(150, 128, 3000, scale=scale, ignored=0.1)
    best = (x.float() @ w.float().T).argmax(-1)
    t = torch.where((torch.arange(150, device=DEV) % 2 == 0) & (t >= 0), best, t)
    got = rl.cross_entropy_forward(x, w, t, softcap=cap, gradient=True)
    check(got, x, w, t, cap=cap)
    assert torch.isfinite(got[2].float()).all()


def test_one_piece_far_above_the_others():
    """One word's logit far above all others, in the first, a middle or the last piece."""
    x, w, t, _ = make(96, 64, 1111, scale=0.1, ignored=0.0)
    for i, v in enumerate((0, 127, 128, 600, 1110)):
        x[i] = 8 * torch.sign(w[v].float()).bfloat16()
        w[v] = 8 * torch.sign(w[v].float()).bfloat16()
    check(rl.cross_entropy_forward(x, w, t, gradient=True), x, w, t)


def test_targets_beyond_and_nothing_to_count():
    x, w, t, weights = make(40, 64, 300, ignored=0.5)
    none = torch.full_like(t, -1)
    loss, losses, dx = rl.cross_entropy_forward(x, w, none, gradient=True)
    assert loss == 0 and torch.all(losses == 0) and torch.all(dx == 0)
    zero = torch.zeros_like(weights)
    got = rl.cross_entropy_forward(x, w, t, weights=zero, gradient=True)
    assert got[0] == 0 and torch.all(got[2] == 0)
    check(got, x, w, t, zero)
    bad = t.clone()
    bad[7] = 300
    loss, losses, dx = rl.cross_entropy_forward(x, w, bad, gradient=True)
    others = torch.arange(40, device=DEV) != 7
    assert torch.isnan(loss) and torch.isnan(losses[7]) and torch.isnan(dx[7].float()).all()
    assert torch.isfinite(losses[others]).all() and torch.isfinite(dx[others].float()).all()
    loss, losses, dx = rl.cross_entropy_forward(x[:0], w, t[:0], gradient=True)
    assert loss == 0 and losses.shape == (0,) and dx.shape == (0, 64)
    # weights of tokens that do not count are not read into anything
    weights[t < 0] = float("nan")
    check(rl.cross_entropy_forward(x, w, t, weights=weights, gradient=True), x, w, t,
          torch.where(t < 0, 0.0, weights))
    # a NaN in one token stays there
    x[3, 5] = float("nan")
    t[3] = 1
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True)
    others = torch.arange(40, device=DEV) != 3
    assert torch.isnan(losses[3]) and torch.isfinite(losses[others]).all()
    assert torch.isfinite(dx[others].float()).all() and torch.isnan(dx[3].float()).any()


def test_strides_shapes_and_place():
    g = torch.Generator(device=DEV).manual_seed(4)
    base = torch.randn(6, 50, 96, generator=g, device=DEV).bfloat16()
    wide = torch.randn(777, 128, generator=g, device=DEV).bfloat16()
    x, w = base[:, :, 8:72], wide[:, 32:96]
    t = torch.randint(-1, 777, (6, 50), generator=g, device=DEV)
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True)
    assert losses.shape == t.shape and dx.shape == x.shape
    flat = lambda a: a.reshape(-1, a.shape[-1]).contiguous()
    check((loss, losses.view(-1), flat(dx)), flat(x), w.contiguous(), t.view(-1))
    # in place, and into a strided output
    room = torch.full((6, 50, 80), 3.0, device=DEV).bfloat16()
    rl.cross_entropy_forward(x, w, t, dX=room[:, :, :64])
    assert torch.equal(room[:, :, :64], dx) and torch.all(room[:, :, 64:] == 3.0)
    y = x.contiguous()
    assert rl.cross_entropy_forward(y, w, t, dX=y)[2] is y and torch.equal(y, dx)
    assert torch.equal(base[:, :, 8:72], x)
    with pytest.raises(ValueError):
        rl.cross_entropy_forward(base[:, ::2, :64][:, :20], w, t[:, :20])
    with pytest.raises(ValueError):
        rl.cross_entropy_forward(x, w, t.view(-1))
    with pytest.raises(TypeError):
        rl.cross_entropy_forward(x.float(), w, t)


def rows_in_64_bits(x, w, t, g, rows):
    """(losses, dX) of a few rows, on the GPU in fp64."""
    z = x[rows].double() @ w.double().T
    p = torch.softmax(z, -1)
    at = torch.arange(len(rows), device=DEV)
    losses = torch.logsumexp(z, -1) - z[at, t[rows]]
    p[at, t[rows]] -= 1
    return losses, (p @ w.double()) * g, (p.abs() @ w.double().abs()) * g


@pytest.mark.parametrize("rows,dim,vocab", [
    (5000, 64, 128001),    # three strips, the last short
    (2048, 4096, 16384),   # 64 tiles of the second product: tails on the spare pairs
    (256, 2048, 20000),    # 4 tiles: cut into ranges
    (2816, 4096, 9001),    # 88 tiles: a whole round, and 12 cut ones
    (6000, 8192, 2100),    # several rounds
])
def test_strips_and_ranges(rows, dim, vocab):
    """Rows from the strips' and tiles' edges; the bound in the mean: U and the products'
    rounding are below 2^-7 of sum |q W|, zerr below 1e-4."""
    x, w, t, _ = make(rows, dim, vocab, ignored=0.0)
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True)
    pick = sorted({0, 1, 127, 128, 255, rows // 2, rows - 1} | {r for r in (2047, 2048, 4095, 4096) if r < rows})
    pick = torch.tensor([r for r in pick if r < rows], device=DEV)
    want, d, size = rows_in_64_bits(x, w, t, 1.0 / rows, pick)
    assert torch.all((losses[pick].double() - want).abs() <= 1e-4 * (1 + want))
    assert torch.all((dx[pick].double() - d).abs() <= 2.0 ** -7 * (size + d.abs()))
    assert abs(float(loss) - float(losses.double().mean())) <= 1e-6 * float(loss)
    # tokens left out do not move the others by more than their factor
    u = t.clone()
    u[::3] = -1
    less = rl.cross_entropy_forward(x, w, u, gradient=True, reduction="sum")
    keep = u >= 0
    assert torch.equal(less[1][keep], losses[keep]) and torch.all(less[1][~keep] == 0)
    assert torch.all(less[2][~keep] == 0)
    near = less[2][keep].double() / rows - dx[keep].double()
    assert float(near.norm() / dx[keep].double().norm()) <= 2.0 ** -8
    rl.device_status()


def test_autograd():
    x, w, t, weights = make(60, 128, 900)
    leaf = x.clone().requires_grad_()
    loss, losses = rl.cross_entropy(leaf.view(6, 10, 128), w, t.view(6, 10), weights=weights.view(6, 10))
    (4.0 * loss).backward()
    _, _, dx = rl.cross_entropy_forward(x, w, t, weights=weights, gradient=True)
    assert torch.equal(leaf.grad, (4.0 * dx.float()).bfloat16())  # a power of two: exact
    assert not losses.requires_grad
    leaf.grad = None
    (loss2, _) = rl.cross_entropy(leaf, w, t, weights=weights)
    (0.3 * loss2).backward()
    assert torch.all((leaf.grad.double() - 0.3 * dx.double()).abs() <= 2.0 ** -8 * 0.301 * dx.double().abs())
    # strides that the kernels do not take are copied
    z = x.t().contiguous().t().requires_grad_()
    rl.cross_entropy(z, w, t, weights=weights)[0].backward()
    assert torch.equal(z.grad, dx)
    odd = torch.empty(60 * 128 + 1, device=DEV, dtype=torch.bfloat16)[1:].view(60, 128).copy_(x).requires_grad_()
    rl.cross_entropy(odd, w, t, weights=weights)[0].backward()
    assert torch.equal(odd.grad, dx)
    with torch.no_grad():
        assert torch.equal(rl.cross_entropy(leaf, w, t, weights=weights)[0], loss2)
    head = w.clone().requires_grad_()
    with pytest.raises(RuntimeError):
        rl.cross_entropy(leaf, head, t)[0].backward()


def test_graph_and_stream():
    x, w, t, _ = make(300, 256, 2000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rl.cross_entropy_forward(x, w, t, gradient=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True)
    for shift in (0, 7):
        t.copy_(torch.where(t >= 0, (t + shift) % 2000, torch.roll(t, shift)))  # other tokens count
        graph.replay()
        want = rl.cross_entropy_forward(x, w, t, gradient=True)
        assert torch.equal(loss, want[0]) and torch.equal(losses, want[1]) and torch.equal(dx, want[2])
    side.wait_stream(torch.cuda.current_stream())
    got = rl.cross_entropy_forward(x, w, t, gradient=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[2], dx)


@pytest.mark.parametrize("rows", [5, 40, 293])
def test_what_the_workspace_held_before(rows):
    """Capped scores: rows behind the last token hold what was there before (here numbers whose scores
    are beyond the cap, NaN, or nothing); the tokens beside them have the same bits."""
    x, w, t, weights = make(rows, 64, 1300, scale=0.5, ignored=0.0)
    got = []
    for fill in (0x0000, 0x4348, 0x7FC0):  # bf16: 0, 200, NaN
        room = torch.full((64 << 19,), fill, dtype=torch.int16, device=DEV)
        got.append(rl.cross_entropy_forward(x, w, t, weights=weights, softcap=30.0, gradient=True, workspace=room))
    check(got[0], x, w, t, weights, 30.0)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("rows,dim,vocab", [(37, 64, 1000), (300, 1000, 3001), (150, 4096, 2000)])
@pytest.mark.parametrize("weighted", [False, True])
def test_losses_of_exact_scores(rows, dim, vocab, weighted):
    """Scores whose products and sums are exact in fp32 (small whole numbers, scaled by 2^-4), so that
    what a loss may be off by is the exponentials' and the sums' alone.  With F = 2^-24 and Z the largest
    score of a row: u = z log2(e) - ref rounds twice and ref once (3 F (2 Z) / ln 2 in u, 6 F Z relative),
    log2(e) itself is off by F (2 F Z); ex2.approx is off by 4 F; a sum has at most 32 + 2 terms a path in a
    piece of 128, then vocab / 128 pieces and 5 steps of shuffles in whatever order: F each; log1p 4 F
    and the loss's own rounding F."""
    g = torch.Generator(device=DEV).manual_seed(dim)
    few = lambda *s: torch.randint(-1, 2, s, generator=g, device=DEV) * (torch.rand(s, generator=g, device=DEV) < 0.3)
    x, w = (few(rows, dim) / 4).bfloat16(), (few(vocab, dim) / 4).bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    weights = torch.rand(rows, generator=g, device=DEV) if weighted else None
    loss, losses, _ = rl.cross_entropy_forward(x, w, t, weights=weights, gradient=True)
    z = x.double() @ w.double().T
    Z = z.abs().max(-1).values
    at = torch.arange(rows, device=DEV)
    rest = z - z[at, t][:, None]
    rest[at, t] = -float("inf")
    want = torch.log1p(torch.exp(rest).sum(-1))
    F = 2.0 ** -24
    bound = F * (8 * Z + 4 + 34 + vocab / 128 + 5) + 5 * F * want
    assert torch.all((losses.double() - want).abs() <= bound)
    share = torch.ones(rows, device=DEV).double() if weights is None else weights.double()
    total, divisor = (share * want).sum(), share.sum()
    assert abs(float(loss) - float(total / divisor)) <= float((share * (bound + 2 * F * want)).sum() / divisor) + 2 * F * float(loss)
    again = rl.cross_entropy_forward(x, w, t, weights=weights)
    assert torch.equal(again[0], loss) and torch.equal(again[1], losses)


@pytest.mark.parametrize("cap", [0.0, 200.0])
@pytest.mark.parametrize("dim", [1024, 4096, 8192])
@pytest.mark.parametrize("rows,vocab", [(40, 1000), (300, 5003)])
def test_losses_where_all_scores_are_large(rows, vocab, dim, cap):
    """Words whose rows are the same but for the last 16 elements, at scores of some 30: what the tensor
    cores' accumulation cuts off along the way is the same for all of them and for the target, and must
    not show.  The last step of 16 products may cut 2^-22 of the largest score Z off each, twice in a
    difference; the cap's formula is off by 8 F Z, twice (F = 2^-24); the rest as for exact scores."""
    g = torch.Generator(device=DEV).manual_seed(dim + vocab)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    common = r(dim) * dim ** -0.5
    w = common.repeat(vocab, 1)
    w[:, -16:] = r(vocab, 16) * 0.5
    x = common * 30 + r(rows, dim) * 0.3
    x[:, -16:] = r(rows, 16)
    x, w = x.bfloat16(), w.bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, softcap=cap, gradient=True)
    z = x.double() @ w.double().T
    Z = z.abs().max(-1).values
    if cap:
        z = cap * torch.tanh(z / cap)
    at = torch.arange(rows, device=DEV)
    rest = z - z[at, t][:, None]
    rest[at, t] = -float("inf")
    want = torch.log1p(torch.exp(rest).sum(-1))
    F = 2.0 ** -24
    bound = 2 * 2.0 ** -22 * Z + F * ((24 if cap else 8) * Z + 4 + 34 + vocab / 128 + 5) + 5 * F * want
    assert torch.all((losses.double() - want).abs() <= bound)
    assert abs(float(loss) - float(want.mean())) <= float(bound.mean()) + 2 * F * float(loss)
    check((loss, losses, dx), x, w, t, cap=cap)


def test_scores_beyond_all_measure():
    """Scores of 1e8 and 1e30, whose last bits are more than the exponentials' range: certain targets
    lose nothing, hopeless ones the difference of the scores; nothing is NaN.  Infinite ones are."""
    w = torch.zeros(300, 64, device=DEV)
    w[7], w[8] = 1.0, -1.0
    x = torch.ones(4, 64, device=DEV) * torch.tensor([1.7e6, 1.7e28, 1.7e6, 1.7e28], device=DEV)[:, None]
    x, w = x.bfloat16(), w.bfloat16()
    t = torch.tensor([7, 7, 8, 8], device=DEV)
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True)
    gap = 128 * x[2:, 0].double()
    assert torch.all(losses[:2] == 0) and torch.all(dx[:2] == 0)
    assert torch.all((losses[2:].double() - gap).abs() <= 2.0 ** -22 * gap)
    want = (w[7] - w[8]).float() / 4
    assert torch.all((dx[2:].float() - want).abs() <= 2.0 ** -7 * want.abs())
    x[1, 3] = float("inf")
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True)
    assert torch.isnan(losses[1]) and torch.isfinite(losses[[0, 2, 3]]).all()
    one = rl.cross_entropy_forward(x[1:2], w[:1], torch.zeros(1, dtype=torch.int64, device=DEV))
    assert torch.isnan(one[1]).all()
