"""The attention block of examples/attention_block_step.py: LoRA layers, rotary
positions, attention and clipping together (needs a GB300).

Gradients are compared in the 2-norm with the same block in 64 bits on the
CPU.  Every bf16 rounding on the way is off by 2^-9 / sqrt(3) of the value's
size in the mean (about 0.0017 in the 2-norm with values spread over a binade);
a gradient passes about 14 of them, each a sum of independent errors: 0.0064,
doubled for the cancellation inside dP - delta, and that three times over as
the bound: 0.04.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "attention_block_step.py")
spec = importlib.util.spec_from_file_location("attention_block_step", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

DEV = "cuda:0"


def reference(block, x, positions, documents, dy):
    """Gradients of the adapters in 64 bits (plain torch on the CPU)."""
    p = {n: {m: getattr(block, m)[n].detach().double().cpu() for m in "WAB"} for n in example.NAMES}
    leaves = {(n, m): p[n][m].requires_grad_() for n in example.NAMES for m in "AB"}
    s = block.alpha / block.A["q"].shape[0]
    lin = lambda n, t: t @ p[n]["W"].T + s * (t @ p[n]["A"].T) @ p[n]["B"].T
    x = x.double().cpu()
    b, n, _ = x.shape
    heads, kvh, d = block.heads, block.kv_heads, block.dim

    def turn(t):
        a = positions.double().cpu()[..., None, None] * torch.tensor(block.freqs.radians,
                                                                     dtype=torch.float64)
        u, w = t[..., :d // 2], t[..., d // 2:]
        return torch.cat((u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()), -1)

    q = turn(lin("q", x).view(b, n, heads, d))
    k = turn(lin("k", x).view(b, n, kvh, d)).repeat_interleave(heads // kvh, 2)
    v = lin("v", x).view(b, n, kvh, d).repeat_interleave(heads // kvh, 2)
    z = torch.einsum("bihd,bjhd->bhij", q, k) * d ** -0.5
    if block.softcap:
        z = block.softcap * torch.tanh(z / block.softcap)
    docs = documents.cpu()
    see = (docs[:, :, None] == docs[:, None]) & (docs[:, :, None] >= 0) & \
        torch.ones(n, n, dtype=torch.bool).tril()
    pr = torch.softmax(z.masked_fill(~see[:, None], -1e300), -1) * see[:, None]
    o = torch.einsum("bhij,bjhd->bihd", pr, v).flatten(2)
    lin("o", o).backward(dy.double().cpu())
    return leaves


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_adapter_gradients(softcap):
    block = example.AttentionBlock(width=256, heads=4, kv_heads=2, rank=8, softcap=softcap, seed=3)
    documents, positions = example.packed([100, 71, 20], 9, DEV)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 200, 256, generator=g).bfloat16().to(DEV)
    dy = torch.randn(1, 200, 256, generator=g).bfloat16().to(DEV)
    block.forward(x, positions, documents).backward(dy)
    rl.device_status()
    leaves = reference(block, x, positions, documents, dy)
    for (n, m), t in leaves.items():
        got = getattr(block, m)[n].grad.double().cpu()
        err = float((got - t.grad).norm() / t.grad.norm())
        assert err <= 0.04, f"d{m} of {n}: {err:.4f}"
    # the clip sees the same gradients
    grads = [t.grad for t in block.adapters]
    want = float(np.sqrt(sum(float(t.double().square().sum()) for t in grads)))
    was = [t.clone() for t in grads]
    norm = rl.GradClip(grads).clip(want / 2)
    assert abs(norm.item() - want) <= 2.0 ** -19 * want
    for t, w in zip(grads, was):
        assert torch.allclose(t.float(), w.float() * 0.5, rtol=2.0 ** -7, atol=0)


def test_the_example_runs():
    losses, apart = example.main(steps=4, tokens=512)
    assert losses[-1] < losses[0]
    assert apart <= 0.02  # two roundings of P and o apart, through one product
