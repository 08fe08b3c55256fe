"""Clipping's plan refuses outputs that share memory with another tensor, on the CPU:
addresses only."""
import numpy as np
import pytest

import test_block_ops_abi_cpu as abi
from rank_linear_gb300 import _lib
from test_block_ops_abi_cpu import BAD, FAKE

BF, F32 = _lib.LORA_BF16, _lib.LORA_FP32


def setup_module():
    abi.setup_module()


def build(*tensors):
    t = (_lib.ClipTensor * len(tensors))(*(_lib.ClipTensor(*x) for x in tensors))
    n = abi.L.lora_clip_plan_bytes(t, len(tensors))
    assert n > 0
    image = np.zeros(n, np.uint8)
    return abi.L.lora_clip_plan_build(t, len(tensors), image.ctypes.data, n)


@pytest.mark.parametrize("tensors", [
    [(FAKE, FAKE, 100, BF), (FAKE, FAKE, 100, BF)],                        # one gradient twice
    [(FAKE, FAKE, 100, BF), (FAKE + 198, FAKE + 198, 1, BF)],              # the last element of another
    [(FAKE, 2 * FAKE, 100, BF), (3 * FAKE, 2 * FAKE + 100, 100, BF)],      # two outputs
    [(FAKE, 2 * FAKE, 100, F32), (2 * FAKE + 396, 3 * FAKE, 100, F32)],    # an output and another's input
    [(2 * FAKE, 3 * FAKE, 1000, BF), (FAKE, 2 * FAKE + 500, 4, F32)],      # within another's input
    [(FAKE, FAKE + 16, 100, BF)],                                          # an output and its own input, shifted
    [(4 * FAKE, 4 * FAKE, 8, BF), (FAKE, FAKE, 1 << 20, F32), (FAKE + 64, 5 * FAKE, 4, BF)],
])
def test_shared_memory(tensors):
    for order in (tensors, tensors[::-1]):
        assert build(*order) == BAD
        assert "shares memory" in abi.L.lora_last_error().decode()


@pytest.mark.parametrize("tensors", [
    [(FAKE, FAKE, 100, BF), (FAKE + 200, FAKE + 200, 100, BF)],            # side by side
    [(FAKE, 2 * FAKE, 100, BF), (FAKE, 2 * FAKE + 200, 100, BF)],          # one input, two outputs
    [(FAKE, 2 * FAKE, 100, BF), (FAKE + 10, 3 * FAKE, 100, BF)],           # inputs that share memory
    [(FAKE, FAKE, 0, BF), (FAKE, FAKE, 5, BF), (None, None, 0, F32)],      # one of nothing
    [],
])
def test_memory_of_its_own(tensors):
    assert build(*tensors) == _lib.LORA_OK
