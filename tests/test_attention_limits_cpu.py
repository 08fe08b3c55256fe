"""Refusals of the attention entry points for what their kernels cannot number or
address, on the CPU: nothing is launched."""
import ctypes

import pytest

import test_block_ops_abi_cpu as abi
from rank_linear_gb300 import _lib
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


TWO = dict(batch=2, q_len=10, k_len=20, q_heads=4, k_heads=2, dim=64)


@pytest.mark.parametrize("at", [0, 1, 2])
def test_broadcast_tensors_of_maps_and_outputs(at):
    """A tensor map's strides are not 0, and an output's entries have a place each."""
    for name, heads in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("d_o", 4), ("dq", 4), ("dk", 2), ("dv", 2)):
        strides = [20 * heads * 64, heads * 64, 64]
        strides[at] = 0
        kw = dict(TWO, **{name: tuple(strides)})
        if name in ("q", "k", "v", "o"):
            assert forward(dict(n=1 << 40), **kw) == UNSUP, name
            assert "broadcast" in abi.L.lora_last_error().decode()
        if name != "o":
            assert backward(dict(n=1 << 40), **kw) == UNSUP, name
            assert "broadcast" in abi.L.lora_last_error().decode()
    assert token(**dict(TWO, q_len=1, o=(0, 64, 64))) == UNSUP


def test_strides_of_single_entries_are_free():
    """Dimensions of one entry: their strides are never used (the workspace is refused next)."""
    one = dict(batch=1, q_len=1, k_len=1, q_heads=1, k_heads=1)
    kw = {n: (0, 0, 0) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")}
    assert backward(dict(n=0), **one, **kw) == _lib.LORA_ERR_WORKSPACE


@pytest.mark.parametrize("at", [0, 1, 2])
def test_broadcast_rotary_outputs(at):
    strides = [2560, 256, 64]
    strides[at] = 0
    assert abi.rotary(q_out=tuple(strides)) == _lib.LORA_ERR_INVALID_ARG
    assert abi.rotary(p_q_out=FAKE, q_in=tuple(strides), q_out=tuple(strides)) == _lib.LORA_ERR_INVALID_ARG
    assert "broadcast" in abi.L.lora_last_error().decode()
