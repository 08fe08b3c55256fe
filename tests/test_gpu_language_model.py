"""The blocks and head of examples/language_model_step.py: norm, dropout, fp8 and bf16
LoRA layers and the loss together (needs a GB300).

Gradients are compared in the 2-norm with the same model in 64 bits on the CPU, whose
fp8 products take the same quantised rows.  On the way a gradient passes, for each
of two blocks, some ten bf16 roundings (2^-9 / sqrt(3) in the mean each, 0.0011 of
its size) and one e4m3 rounding of dY (2^-4 / sqrt(3) = 0.036 of each element,
independent ones, which the products' sums keep at that size); the activations'
e4m3 rounding is in the reference.  Together 2^(1/2) 0.036 + 20^(1/2) 0.0011 = 0.056,
with a factor of 1.5 for cancellation: 0.085.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import norm as on

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "language_model_step.py")
spec = importlib.util.spec_from_file_location("language_model_step", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

DEV = "cuda:0"


class Quantised(torch.autograd.Function):
    """y as its e4m3 rows stand for it; the gradient as it comes."""

    @staticmethod
    def forward(ctx, y):
        scale = torch.from_numpy(on.row_scale(y.numpy()))[:, None]
        return (y / scale).to(torch.float32).to(torch.float8_e4m3fn).double() * scale

    @staticmethod
    def backward(ctx, d):
        return d


def reference(model, tokens, targets, seed, train=True):
    """(loss, gradients) with plain torch in 64 bits on the CPU."""
    d = lambda t: t.detach().double().cpu()
    params = [d(t).requires_grad_() for t in model.parameters()]
    norms = params[:len(model.norms)]
    rest = iter(params[len(model.norms):])
    tokens, targets = tokens.cpu().flatten(), targets.cpu().flatten()
    keep = lambda n, c, off: torch.from_numpy(on.dropout(np.ones((n, c)), model.p if train else 0.0, seed, off))

    def norm(h, w):
        return h * (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w

    s = model.alpha / model.adapters[0][0].shape[0]
    h, branch, n = d(model.embed)[tokens], None, len(tokens)
    for i in range(len(model.adapters)):
        a_up, b_up, a_down, b_down = (next(rest) for _ in range(4))
        if branch is not None:
            h = h + branch * keep(n, h.shape[1], i)
        y = norm(h, norms[i])
        q = model.up_q[i]
        w = q.Wq.view(torch.float8_e4m3fn).float().double().cpu() * q.w_scale.double().cpu()
        u = Quantised.apply(y) @ w.T + s * (y @ a_up.T) @ b_up.T
        u = u * keep(n, u.shape[1], 100 + i)
        branch = u @ d(model.down_w[i]).T + s * (u @ a_down.T) @ b_down.T
    h = h + branch * keep(n, h.shape[1], len(model.adapters))
    z = norm(h, norms[-1]) @ d(model.head).T
    if model.softcap:
        z = model.softcap * torch.tanh(z / model.softcap)
    live = targets >= 0
    loss = -(torch.log_softmax(z, -1)[torch.arange(n), targets.clamp(min=0)] * live).sum() / live.sum()
    loss.backward()
    return loss.item(), [p.grad for p in params]


@pytest.mark.parametrize("softcap", [0.0, 4.0])
def test_gradients(softcap):
    model = example.Model(vocab=1003, softcap=softcap, seed=2)
    g = torch.Generator().manual_seed(3)
    tokens = torch.randint(0, 1003, (2, 75), generator=g).to(DEV)
    targets = torch.roll(tokens, -1, 1)
    targets[0, :30] = -100
    loss, each = model.loss(tokens, targets, seed=11)
    loss.backward()
    rl.device_status()
    want, grads = reference(model, tokens, targets, 11)
    assert abs(loss.item() - want) <= 0.02 * want and torch.all(each[0, :30] == 0)
    for t, w in zip(model.parameters(), grads):
        err = float((t.grad.double().cpu() - w).norm() / w.norm())
        assert err <= 0.085, f"{tuple(t.shape)}: {err:.4f}"


def test_captured_step():
    """Forward and backward in one graph, replayed with other masks and tokens."""
    model = example.Model(vocab=1003, seed=4)
    words = torch.tensor([5, 0], device=DEV)
    tokens = torch.randint(0, 1003, (2, 64), device=DEV)
    targets = torch.roll(tokens, -1, 1)

    def step():
        loss, _ = model.loss(tokens, targets, words)
        return (loss,) + torch.autograd.grad(loss, model.parameters())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (5, 6):
        words.copy_(torch.tensor([seed, 0]))
        tokens.copy_(torch.roll(tokens, 3, 0))
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
    rl.device_status()


def test_the_example_runs():
    losses, score = example.main(steps=3, tokens=128)
    assert all(np.isfinite(losses)) and np.isfinite(score) and score < 0
