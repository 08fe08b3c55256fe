"""Refusals of the attention entry points for what their kernels cannot number or
address, on the CPU: nothing is launched."""
import ctypes

import pytest

import test_block_ops_abi_cpu as abi
from test_block_ops_abi_cpu import FAKE, UNSUP, backward, forward, shape


def setup_module():
    abi.setup_module()


def token(**kw):
    s = shape(**dict(dict(q_len=1, causal=0), **kw))
    return abi.L.lora_attention_token(ctypes.byref(s), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 62, None)


# batch * q_heads * tiles above 2^30 (the last: not), within the limit of rows
MANY = [dict(batch=32769, q_heads=32768, k_heads=1, q_len=1, k_len=1),
        dict(batch=65535, q_heads=43690, k_heads=1, q_len=1, k_len=1),
        dict(batch=32768, q_heads=65535, k_heads=1, q_len=0, k_len=1),
        dict(batch=16384, q_heads=32768, k_heads=32768, q_len=1, k_len=14)]


@pytest.mark.parametrize("kw", MANY[:3])
def test_more_tiles_than_their_numbers_hold(kw):
    kw = dict(kw, dim=8, causal=0)
    assert forward(dict(n=1 << 62), **kw) == UNSUP
    assert backward(dict(n=1 << 62), **kw) == UNSUP
    assert "tiles" in abi.L.lora_last_error().decode()
    assert abi.L.lora_attention_workspace_bytes(ctypes.byref(shape(**kw)), 1) == 0
    if kw["q_len"] == 1:
        assert token(**kw) == UNSUP


def test_as_many_tiles_as_their_numbers_hold():
    s = shape(**dict(MANY[3], dim=8, causal=0))
    assert abi.L.lora_attention_workspace_bytes(ctypes.byref(s), 1) > 0
    s = shape(batch=32768, q_heads=32768, k_heads=1, q_len=1, k_len=1, dim=8, causal=0)
    assert abi.L.lora_attention_workspace_bytes(ctypes.byref(s), 1) > 0
