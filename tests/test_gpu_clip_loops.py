"""Clipping in training loops that clear, drop or replace their gradients (needs a
GB300)."""
import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def layers():
    torch.manual_seed(0)
    return [torch.randn(64, 32, device=DEV).requires_grad_(), torch.randn(16, 32, device=DEV).requires_grad_()]


def backward(params, x):
    sum((p * x).square().sum() for p in params).backward()


def norm_of(tensors):
    return torch.cat([t.double().flatten() for t in tensors]).norm().item()


def test_gradients_cleared_in_place():
    params = layers()
    opt = torch.optim.SGD(params, lr=0.01)
    backward(params, 1.0)
    clip = rl.GradClip(params=params)
    for step in range(3):
        opt.zero_grad(set_to_none=False)
        backward(params, 1.0 + step)
        want = norm_of([p.grad for p in params])
        got = clip.clip(0.5).item()
        assert abs(got - want) <= 2.0 ** -19 * want
        assert abs(norm_of([p.grad for p in params]) - 0.5) <= 1e-5
        opt.step()


def test_gradients_dropped_and_made_again():
    """zero_grad() as it is by default: the plan does not clip what is not in use."""
    params = layers()
    opt = torch.optim.SGD(params, lr=0.01)
    backward(params, 1.0)
    clip = rl.GradClip(params=params)
    first = [p.grad.clone() for p in params]
    old = [p.grad for p in params]
    opt.zero_grad()
    with pytest.raises(RuntimeError, match="gradient"):
        clip.clip(0.5)
    backward(params, 2.0)
    for call in (lambda: clip.clip(0.5), clip.norm):
        with pytest.raises(RuntimeError, match="gradient"):
            call()
    for a, b in zip(old, first):
        assert torch.equal(a, b)
    clip = rl.GradClip(params=params)
    want = norm_of([p.grad for p in params])
    assert abs(clip.clip(0.5).item() - want) <= 2.0 ** -19 * want
    params[1].grad = params[1].grad.clone()
    with pytest.raises(RuntimeError, match="parameter 1"):
        clip.clip(0.5)


def test_gradients_with_their_parameters():
    params = layers()
    backward(params, 1.0)
    out = [torch.empty_like(p) for p in params]
    clip = rl.GradClip([p.grad for p in params], out=out, params=params)
    want = norm_of([p.grad for p in params])
    assert abs(clip.clip(0.5).item() - want) <= 2.0 ** -19 * want
    assert abs(norm_of(out) - 0.5) <= 1e-5
    with pytest.raises(ValueError):
        rl.GradClip([p.grad for p in params], params=params[:1])
    with pytest.raises(RuntimeError, match="parameter 0"):
        rl.GradClip([p.grad.clone() for p in params], params=params)
    params[0].grad = None
    with pytest.raises(ValueError):
        rl.GradClip(params=params)
    with pytest.raises(ValueError):
        rl.GradClip()


def test_memory_of_the_plan_stays_its_own():
    """A gradient that is given other memory leaves the old to the plan, not to the
    next tensor that is made."""
    g = torch.ones(1 << 20, device=DEV)
    clip = rl.GradClip([g])
    place = g.data_ptr()
    g.data = torch.ones(1 << 20, device=DEV)
    others = [torch.full((1 << 20,), 3.0, device=DEV) for _ in range(8)]
    assert all(t.data_ptr() != place for t in others)
    clip.clip(0.5)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in others) and bool((g == 1).all())
