"""Attention where it can go wrong beyond the usual sizes and values: waits between
the warps of a block, extreme caps, few visible keys among many, tensors that the
kernels cannot take as they are (needs a GB300).

The reference and its bounds are those of test_gpu_attention.py.
"""
import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from test_gpu_attention import DEV, check, draw

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
