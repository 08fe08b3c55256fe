"""Refusals of the rotary, attention and clip entry points, on the CPU: every
argument is checked before anything touches CUDA (no launches)."""
import ctypes
import math

import numpy as np
import pytest

from oracle import attention as oa
from rank_linear_gb300 import _lib, build

FAKE = 0x100000  # aligned non-null "device" address; never dereferenced here
BAD, UNSUP, WS = _lib.LORA_ERR_INVALID_ARG, _lib.LORA_ERR_UNSUPPORTED, _lib.LORA_ERR_WORKSPACE
L = None


def setup_module():
    global L
    build.build()
    L = _lib.lib()


def rotary(**kw):
    a = dict(q=FAKE, k=FAKE, pos=FAKE, turns=FAKE, dt=_lib.LORA_BF16, q_out=2 * FAKE, k_out=2 * FAKE)
    sh = dict(batch=2, seq=10, q_heads=4, k_heads=2, dim=64, rot=64, position_bits=64,
              magnitude=1.0, q_in=(2560, 256, 64), q_out=(2560, 256, 64), k_in=(1280, 128, 64),
              k_out=(1280, 128, 64), position=(10, 1))
    for n, v in kw.items():
        if n.startswith("p_"):
            a[n[2:]] = v
        else:
            sh[n] = v
    s = _lib.RotaryShape(**sh)
    return L.lora_rotary(ctypes.byref(s), a["q"], a["k"], a["pos"], a["turns"], a["dt"],
                         a["q_out"], a["k_out"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), BAD), (dict(seq=-1), BAD), (dict(q_heads=-1), BAD), (dict(rot=63), BAD),
    (dict(rot=66), BAD), (dict(rot=0), BAD), (dict(dim=2048, rot=64), BAD),
    (dict(interleaved=2), BAD), (dict(inverse=-1), BAD), (dict(position_bits=16), BAD),
    (dict(magnitude=math.nan), BAD), (dict(p_q=None), BAD), (dict(p_k_out=None), BAD),
    (dict(p_pos=None), BAD), (dict(p_turns=FAKE + 4), BAD), (dict(p_pos=FAKE + 4), BAD),
    (dict(p_q=FAKE + 1), BAD), (dict(p_dt=5), BAD),
    (dict(p_q_out=FAKE, q_out=(2560, 64, 640)), BAD),      # in place with other strides
    (dict(seq=1 << 32), UNSUP), (dict(seq=1 << 30, q_heads=65536), UNSUP),
])
def test_rotary_rejects(kw, code):
    assert rotary(**kw) == code
    assert L.lora_last_error().decode() != ""


def test_rotary_nothing_to_do():
    assert rotary(seq=0, p_q=None, p_k=None, p_pos=None, p_turns=None) == _lib.LORA_OK
    assert rotary(q_heads=0, k_heads=0) == _lib.LORA_OK


def test_rotary_turns():
    w = [1.0, 0.5, -1.0, 2 * math.pi, 1e-9, 0.0, 100.0]
    out = (ctypes.c_uint64 * len(w))()
    assert L.lora_rotary_turns((ctypes.c_double * len(w))(*w), len(w), out) == _lib.LORA_OK
    for x, t in zip(w, out):
        got = t / 2.0 ** 64
        want = (x / (2 * math.pi)) % 1.0
        d = abs(got - want)
        assert min(d, 1.0 - d) <= 2.0 ** -46
    assert L.lora_rotary_turns(None, 1, out) == BAD
    assert L.lora_rotary_turns((ctypes.c_double * 1)(math.inf), 1, out) == BAD
    assert L.lora_rotary_turns(None, -1, None) == BAD


def test_clip_plan():
    t = (_lib.ClipTensor * 2)(_lib.ClipTensor(FAKE, FAKE, 5000, _lib.LORA_BF16),
                              _lib.ClipTensor(None, None, 0, _lib.LORA_FP32))
    n = L.lora_clip_plan_bytes(t, 2)
    assert n > 0
    # 5000 bf16 in 4 KB chunks: 3 records of 32 bytes
    empty = L.lora_clip_plan_bytes(t, 0)
    assert n - empty == 3 * 32
    image = np.zeros(n, np.uint8)
    assert L.lora_clip_plan_build(t, 2, image.ctypes.data, n) == _lib.LORA_OK
    assert L.lora_clip_plan_build(t, 2, image.ctypes.data, n - 1) == WS
    assert L.lora_clip_plan_build(t, 2, None, n) == WS
    records = image[empty:].view(np.int64).reshape(3, 4)
    assert records[:, 0].tolist() == [FAKE, FAKE + 4096, FAKE + 8192]
    assert (records[:, 2] & 0xffffffff).tolist() == [2048, 2048, 904]


@pytest.mark.parametrize("tensor", [
    (None, FAKE, 4, 0), (FAKE, None, 4, 0), (FAKE + 1, FAKE, 4, 0), (FAKE, FAKE + 2, 4, 1),
    (FAKE, FAKE, -1, 0), (FAKE, FAKE, 4, 3)])
def test_clip_plan_rejects(tensor):
    t = (_lib.ClipTensor * 1)(_lib.ClipTensor(*tensor))
    assert L.lora_clip_plan_bytes(t, 1) == 0
    assert L.lora_last_error().decode() != ""


@pytest.mark.parametrize("args", [
    (None, 1 << 16, 1.0, 0, FAKE), (FAKE, 1 << 16, 1.0, 0, None), (FAKE + 8, 1 << 16, 1.0, 0, FAKE),
    (FAKE, 100, 1.0, 0, FAKE), (FAKE, (1 << 16) + 8, 1.0, 0, FAKE), (FAKE, 32784, 1.0, 2, FAKE),
    (FAKE, 32784, -1.0, 0, FAKE), (FAKE, 32784, math.nan, 0, FAKE), (FAKE, 32784, 1.0, 0, FAKE + 2)])
def test_clip_rejects(args):
    assert L.lora_clip(*args, None) == BAD
    assert L.lora_last_error().decode() != ""


def shape(**kw):
    a = dict(batch=1, q_len=10, k_len=20, q_heads=4, k_heads=2, dim=64, causal=1, scale=0.125)
    for n, h in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("d_o", 4), ("dq", 4), ("dk", 2), ("dv", 2)):
        a[n] = (20 * h * 64, h * 64, 64)
    a.update(kw)
    return _lib.AttentionShape(**a)


def forward(ptr=None, **kw):
    s = shape(**kw)
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, ws=FAKE, n=1 << 30)
    a.update(ptr or {})
    return L.lora_attention_fwd(ctypes.byref(s), a["q"], a["k"], a["v"], a["o"], a["lse"], a["ws"],
                                a["n"], None)


def backward(ptr=None, **kw):
    s = shape(**kw)
    a = dict(d_o=FAKE, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             ws=FAKE, n=1 << 30)
    a.update(ptr or {})
    return L.lora_attention_bwd(ctypes.byref(s), a["d_o"], a["q"], a["k"], a["v"], a["o"], a["lse"],
                                a["dq"], a["dk"], a["dv"], a["ws"], a["n"], None)


SHAPES = [
    (dict(batch=-1), BAD), (dict(q_len=-1), BAD), (dict(q_heads=3), BAD), (dict(k_heads=0), BAD),
    (dict(dim=0), BAD), (dict(dim=60), UNSUP), (dict(dim=136), UNSUP), (dict(causal=2), BAD),
    (dict(scale=math.inf), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(softcap=-1.0), BAD), (dict(softcap=math.nan), BAD),
    (dict(q_docs=FAKE), BAD), (dict(causal=0, prefix=FAKE), BAD), (dict(slopes=FAKE + 2), BAD),
    (dict(k_len=1 << 24), UNSUP), (dict(q=(0, 4 * 64 + 4, 64)), UNSUP),
    (dict(v=(0, -128, 64)), UNSUP),
]


@pytest.mark.parametrize("kw,code", SHAPES)
def test_attention_rejects(kw, code):
    for f in (forward, backward):
        assert f(**kw) == code
        assert L.lora_last_error().decode() != ""


def test_attention_rejects_pointers():
    for n in ("q", "k", "v", "o"):
        assert forward({n: None}) == BAD and forward({n: FAKE + 8}) == BAD
    for n in ("d_o", "q", "k", "v", "o", "lse", "dq", "dk", "dv"):
        assert backward({n: None}) == BAD
    assert backward({"ws": None, "n": 0}) == WS and backward({"n": 16}) == WS
    assert L.lora_attention_fwd(None, *[FAKE] * 6, 0, None) == BAD
    assert L.lora_attention_workspace_bytes(None, 0) == 0


def test_attention_nothing_to_do():
    none = dict(q=None, o=None, lse=None)
    assert forward(none, q_len=0) == _lib.LORA_OK
    assert forward(dict(none, k=None, v=None), batch=0) == _lib.LORA_OK


@pytest.mark.parametrize("kw,ptr,code", [
    (dict(q_len=2), {}, BAD), (dict(causal=1), {}, BAD), (dict(prefix=FAKE), {}, BAD),
    (dict(q_docs=FAKE, k_docs=FAKE), {}, BAD), (dict(dim=12), {}, UNSUP),
    (dict(), {"lengths": None}, BAD), (dict(), {"lengths": FAKE + 1}, BAD),
    (dict(), {"q": None}, BAD), (dict(k=(0, 4, 64)), {}, UNSUP)])
def test_token_rejects(kw, ptr, code):
    s = shape(**dict(dict(q_len=1, causal=0), **kw))
    a = dict(q=FAKE, k=FAKE, v=FAKE, lengths=FAKE, o=FAKE, ws=FAKE, n=1 << 30)
    a.update(ptr)
    assert L.lora_attention_token(ctypes.byref(s), a["q"], a["k"], a["v"], a["lengths"], a["o"],
                                  a["ws"], a["n"], None) == code


@pytest.mark.parametrize("kw", [dict(), dict(cap=3.0), dict(slopes=np.array([0.5, 0.1])),
                                dict(cap=3.0, prefix=[4, 9]),
                                dict(q_docs=np.array([[0, 0, 1, 1, -1, 2, 2, 2]] * 2))])
def test_reference_gradients_against_differences(kw):
    """The 64-bit reference's own gradients are those of its forward pass."""
    rng = np.random.default_rng(1)
    q, do = rng.standard_normal((2, 2, 8, 2, 4))
    k, v = rng.standard_normal((2, 2, 8, 1, 4))
    if "q_docs" in kw:
        kw = dict(kw, k_docs=kw["q_docs"])
    opts = dict(scale=0.7, causal=True, **kw)
    r = oa.run(q, k, v, do, **opts)
    h = 1e-6
    for n, name in enumerate(("dq", "dk", "dv")):
        for _ in range(10):
            x = [q, k, v]
            at = tuple(rng.integers(0, s) for s in x[n].shape)
            step = np.zeros_like(x[n])
            step[at] = h
            f = lambda sign: (oa.run(*[y + sign * step if i == n else y for i, y in enumerate(x)],
                                     **opts)["o"] * do).sum()
            assert abs((f(1) - f(-1)) / (2 * h) - r[name][at]) <= 1e-7
