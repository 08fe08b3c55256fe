"""Norm, dropout and loss where addresses pass 32 bits, where two calls run at once, and
in graphs whose tokens change (needs a GB300)."""
import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def apart(rows, dim, step, t):
    """t [rows, dim] with its rows `step` elements apart in one large allocation."""
    room = torch.empty((rows - 1) * step + dim, dtype=t.dtype, device=DEV)
    out = room.as_strided((rows, dim), (step, 1))
    return out.copy_(t)


@pytest.mark.parametrize("rows,dim,step", [
    (3, 2048, 2 ** 31),       # few rows
    (513, 1536, 2 ** 23),     # over the ring
    (513, 1530, 2 ** 23 + 2),
    (1025, 200, 2 ** 22 + 8),
])
def test_norm_rows_far_apart(rows, dim, step):
    """The same bits as the rows side by side (both take the same kernel)."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    x, res, dy, dh = (torch.randn(rows, dim, generator=g, device=DEV).bfloat16() for _ in range(4))
    w = torch.rand(dim, generator=g, device=DEV).bfloat16()
    opts = dict(dropout=0.25, seed=9)
    near = rl.rms_norm_forward(x, w, residual=res, **opts)
    grads = rl.rms_norm_backward(dy, near[1], w, near[2], dh=dh, **opts)
    far = rl.rms_norm_forward(apart(rows, dim, step, x), w, residual=res, out=apart(rows, dim, step, x), **opts)
    for a, b in zip(near, far):
        assert torch.equal(a, b)
    far = rl.rms_norm_backward(dy, apart(rows, dim, step, near[1]), w, near[2], dh=dh,
                               dx=apart(rows, dim, step, x), **opts)
    for a, b in zip(grads, far):
        assert torch.equal(a, b)
    assert torch.equal(rl.dropout_forward(apart(rows, dim, step, x), 0.25, 9), rl.dropout_forward(x, 0.25, 9))
    rl.device_status()


def test_loss_rows_far_apart():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(33, 64, generator=g, device=DEV).bfloat16()
    w = torch.randn(600, 64, generator=g, device=DEV).bfloat16()
    t = torch.randint(-1, 600, (33,), generator=g, device=DEV)
    near = rl.cross_entropy_forward(x, w, t, gradient=True)
    far = rl.cross_entropy_forward(apart(33, 64, 2 ** 27, x), w, t, dX=apart(33, 64, 2 ** 27, x))
    for a, b in zip(near, far):
        assert torch.equal(a, b)
    far = rl.cross_entropy_forward(x, apart(600, 64, 2 ** 23, w), t, gradient=True)
    for a, b in zip(near, far):
        assert torch.equal(a, b)
    rl.device_status()


def test_loss_of_few_tokens_in_strips():
    """A vocabulary of which 256 tokens fill a strip: four strips, whose tokens each find
    their places by themselves."""
    g = torch.Generator(device=DEV).manual_seed(2)
    vocab = 1_100_003
    x = torch.randn(800, 64, generator=g, device=DEV).bfloat16()
    w = (torch.randn(vocab, 64, generator=g, device=DEV) / 8).bfloat16()
    t = torch.randint(0, vocab, (800,), generator=g, device=DEV)
    t[torch.rand(800, generator=g, device=DEV) < 0.2] = -1
    loss, losses, dx = rl.cross_entropy_forward(x, w, t, gradient=True, reduction="sum")
    rows = torch.tensor([r for r in range(0, 800, 37) if t[r] >= 0], device=DEV)
    z = x[rows].double() @ w.double().T
    p = torch.softmax(z, -1)
    at = torch.arange(len(rows), device=DEV)
    want = torch.logsumexp(z, -1) - z[at, t[rows]]
    p[at, t[rows]] -= 1
    d, size = p @ w.double(), p.abs() @ w.double().abs()
    # (logits' errors below 1e-4; an exponential's rounding and the output's: 2^-8 each)
    assert torch.all((losses[rows].double() - want).abs() <= 1e-4 * (1 + want))
    assert torch.all((dx[rows].double() - d).abs() <= 2.0 ** -7 * (size + d.abs()))
    assert torch.all(losses[t < 0] == 0) and torch.all(dx[t < 0] == 0)
    assert abs(float(loss) - float(losses.double().sum())) <= 1e-6 * float(loss)
    rl.device_status()


@pytest.mark.parametrize("rows", [900, 1500])
def test_loss_graph_whose_tokens_change(rows):
    """Replayed with more, fewer and no tokens that count, and other weights."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, 128, generator=g, device=DEV).bfloat16()
    w = torch.randn(1000, 128, generator=g, device=DEV).bfloat16()
    t = torch.randint(0, 1000, (rows,), generator=g, device=DEV)
    weights = torch.rand(rows, generator=g, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rl.cross_entropy_forward(x, w, t, weights=weights, gradient=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rl.cross_entropy_forward(x, w, t, weights=weights, gradient=True)
    for part in (0.0, 0.7, 1.0, 0.1):
        t.copy_(torch.randint(0, 1000, (rows,), generator=g, device=DEV))
        t[torch.rand(rows, generator=g, device=DEV) < part] = -100
        weights.uniform_(generator=g)
        graph.replay()
        want = rl.cross_entropy_forward(x, w, t, weights=weights, gradient=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    rl.device_status()


def test_calls_at_once():
    """Four streams with calls of their own in flight together: each has the bits that it
    has alone."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(4, 700, 1536, generator=g, device=DEV).bfloat16()
    w = torch.randn(2000, 1536, generator=g, device=DEV).bfloat16()
    scale = torch.rand(1536, generator=g, device=DEV).bfloat16()
    t = torch.randint(-1, 2000, (4, 700), generator=g, device=DEV)

    def step(i):
        y, h, rstd = rl.rms_norm_forward(x[i], scale, residual=x[i - 1], dropout=0.1, seed=i)
        loss, losses, dy = rl.cross_entropy_forward(y, w, t[i], gradient=True)
        dx, dres, dw = rl.rms_norm_backward(dy, h, scale, rstd, dh=x[i], dropout=0.1, seed=i)
        return loss, losses, dx, dres, dw, rl.dropout_forward(dx, 0.5, i)
    alone = [step(i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(3):
        got = []
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step(i))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(alone, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
        torch.cuda.synchronize()
    rl.device_status()


def test_the_same_tensor_twice():
    """x as its own residual, a leaf that is both, and one vector as a row."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(40, 64, generator=g, device=DEV, requires_grad=True)
    w = torch.rand(64, generator=g, device=DEV).add_(0.5).requires_grad_()
    y, h = rl.rms_norm(x, w, residual=x, eps=1e-4)
    (y.sum() + 2 * h.sum()).backward()
    a, b = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    h64 = a + a
    y64 = h64 * (h64.square().mean(-1, keepdim=True) + 1e-4).rsqrt() * b
    (y64.sum() + 2 * h64.sum()).backward()
    assert torch.equal(h, 2 * x)
    assert torch.allclose(x.grad.double(), a.grad, rtol=1e-5, atol=2e-5)
    assert torch.allclose(w.grad.double(), b.grad, rtol=1e-5, atol=2e-5)
    row = rl.rms_norm_forward(x.detach()[3], w.detach(), eps=1e-4)
    many = rl.rms_norm_forward(x.detach()[3:4], w.detach(), eps=1e-4)
    assert row[0].shape == (64,) and row[2].shape == () and torch.equal(row[0], many[0][0])
    head = torch.randn(90, 64, generator=g, device=DEV).bfloat16()
    v = x.detach()[3].bfloat16().requires_grad_()
    loss, one = rl.cross_entropy(v, head, torch.tensor(7, device=DEV))
    loss.backward()
    assert one.shape == () and torch.equal(one, loss.detach()) and v.grad.shape == (64,)


def test_no_gradient_where_none_is_taken():
    """Under no_grad the loss of a leaf costs its first product only."""
    x = torch.randn(20, 64, device=DEV).bfloat16().requires_grad_()
    w, t = torch.randn(50, 64, device=DEV).bfloat16(), torch.arange(20, device=DEV)
    with torch.no_grad():
        loss, losses = rl.cross_entropy(x, w, t)
    assert not loss.requires_grad
    want = rl.cross_entropy_forward(x.detach(), w, t)
    assert want[2] is None and torch.equal(loss, want[0]) and torch.equal(losses, want[1])
