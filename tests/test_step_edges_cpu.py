"""Calls of the loss that are refused: softcaps whose inverse or square leaves fp32, and
losses written over the weights that are still read."""
import ctypes

import pytest
import torch

import rank_linear_gb300 as rl
from rank_linear_gb300 import _lib

L = _lib.lib()
AT = 1 << 20  # an address that is only compared


def call(softcap=0.0, each=6 * AT, weights=4 * AT):
    sh = _lib.LossShape(rows=10, vocab=100, dim=64, target_bits=64, mean=1, softcap=softcap, x=64, w=64, dx=64)
    return L.lora_loss(ctypes.byref(sh), AT, 2 * AT, 3 * AT, weights, 5 * AT, each, 7 * AT, None, 0, None)


@pytest.mark.parametrize("cap", [2.0 ** -101, 1e-45, 2.0 ** 101, 3e38, -2.0 ** -101])
def test_softcaps_out_of_range(cap):
    assert call(softcap=cap) == _lib.LORA_ERR_INVALID_ARG
    assert "softcap" in L.lora_last_error().decode()


@pytest.mark.parametrize("cap", [0.0, 2.0 ** -100, 2.0 ** 100])
def test_softcaps_at_the_ends(cap):
    assert call(softcap=cap) == _lib.LORA_ERR_WORKSPACE  # the next thing that is checked


def test_losses_over_the_weights():
    assert call(each=4 * AT) == _lib.LORA_ERR_INVALID_ARG
    assert call(each=4 * AT, weights=None) == _lib.LORA_ERR_WORKSPACE


@pytest.mark.parametrize("cap", [1e-50, 1e39, -1.0, float("nan"), float("inf")])
def test_softcaps_that_fp32_would_change(cap):
    x, w, t = torch.zeros(4, 8).bfloat16(), torch.zeros(5, 8).bfloat16(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="softcap"):
        rl.cross_entropy_forward(x, w, t, softcap=cap)
