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
