"""What autograd may and may not ask of rotary positions and attention (needs a GB300)."""
import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def draw(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def test_no_gradients_of_gradients():
    """A loss of gradients says that it cannot be had, instead of leaving them out."""
    q, k, v = draw(1, 30, 2, 64).requires_grad_(), draw(1, 30, 1, 64, seed=1), draw(1, 30, 1, 64, seed=2)
    g, = torch.autograd.grad(rl.attention(q, k, v, causal=True).float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (g.float().square().sum() + q.float().square().sum()).backward()
    f = rl.rotary_frequencies(64, device=DEV)
    a, _ = rl.rotary(q, k, torch.arange(30, device=DEV), f)
    g, = torch.autograd.grad(a.float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (g.float().square().sum() + q.float().square().sum()).backward()


def test_slopes_get_no_gradient_and_say_so():
    q, k, v = draw(1, 30, 2, 64).requires_grad_(), draw(1, 30, 1, 64, seed=1), draw(1, 30, 1, 64, seed=2)
    slopes = torch.tensor([0.5, 0.25], device=DEV, requires_grad=True)
    o = rl.attention(q, k, v, causal=True, slopes=slopes)
    with pytest.raises(RuntimeError, match="slopes"):
        o.float().sum().backward()
    with torch.no_grad():
        a = rl.attention(q, k, v, causal=True, slopes=slopes)
    b = rl.attention(q, k, v, causal=True, slopes=slopes.detach())
    b.float().sum().backward()
    assert torch.equal(a, b) and q.grad.isfinite().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotary_of_strided_heads(dtype):
    f = rl.rotary_frequencies(64, device=DEV)
    pos = torch.arange(30, device=DEV)
    x = draw(2, 30, 4, 128).to(dtype)
    q = x[..., ::2].detach().requires_grad_()
    k = draw(2, 30, 64, 2, seed=1).to(dtype).transpose(2, 3).detach().requires_grad_()
    gq, gk = draw(2, 30, 4, 64, seed=2).to(dtype), draw(2, 30, 2, 64, seed=3).to(dtype)
    a, b = rl.rotary(q, k, pos, f)
    torch.autograd.backward((a, b), (gq, gk))
    a1, b1 = rl.rotary_forward(q.detach().contiguous(), k.detach().contiguous(), pos, f)
    dq, dk = rl.rotary_backward(gq, gk, pos, f)
    for got, want in ((a, a1), (b, b1), (q.grad, dq), (k.grad, dk)):
        assert torch.equal(got, want)


def test_gradients_have_memory_of_their_own():
    """Keeping, saving or changing one gradient does nothing with the others."""
    q, k, v = (draw(1, 300, h, 64, seed=s).requires_grad_() for s, h in enumerate((4, 2, 2)))
    rl.attention(q, k, v, causal=True).float().square().sum().backward()
    grads = [t.grad for t in (q, k, v)]
    assert len({g.untyped_storage().data_ptr() for g in grads}) == 3
    for g in grads:
        assert g.untyped_storage().nbytes() <= g.numel() * g.element_size() + 512
    before = [g._version for g in grads]
    grads[0].mul_(0.5)
    assert [g._version for g in grads[1:]] == before[1:]
