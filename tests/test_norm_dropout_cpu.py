"""The generator and the norm's oracle against published and closed values, and the
refusals of the norm and dropout entry points, on the CPU (no launches)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import norm as on
from rank_linear_gb300 import _lib, build

FAKE = 0x100000  # aligned non-null "device" address; never dereferenced here
BAD, UNSUP, WS = _lib.LORA_ERR_INVALID_ARG, _lib.LORA_ERR_UNSUPPORTED, _lib.LORA_ERR_WORKSPACE
L = None


def setup_module():
    global L
    build.build()
    L = _lib.lib()


def test_philox_published_vectors():
    """The known answers that the generator's authors publish."""
    f = 0xFFFFFFFF
    assert on.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert on.philox([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert on.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_words_are_the_generators():
    seed, offset = 0x0123456789ABCDEF, 77
    w = on.words(3, 11, seed, offset, first_row=2 ** 32 - 1)
    for n in range(3):
        row = 2 ** 32 - 1 + n
        for c in range(11):
            want = on.philox([c // 4, row & 0xFFFFFFFF, row >> 32, offset],
                             [seed & 0xFFFFFFFF, seed >> 32])[c % 4]
            assert int(w[n, c]) == want


def test_dropout_keeps_the_expectation():
    x = np.ones((200, 1000))
    for p in (0.0, 0.1, 0.5, 0.9):
        y = on.dropout(x, p, 5, 6)
        share = (y != 0).mean()  # of 200,000: three standard deviations of a binomial
        assert abs(share - (1 - p)) <= 3 * math.sqrt(p * (1 - p) / x.size) + 1e-9
        # T = p 2^32 to half a unit: 1 - T / 2^32 is off by 2^-33, relative to 1 - p
        assert abs(y.max() * (1 - p) - 1) <= 1.01 * 2.0 ** -33 / (1 - p)


def test_norm_oracle_closed_forms_and_differences():
    rng = np.random.default_rng(1)
    h, w, dy = rng.normal(size=(4, 7)), rng.normal(size=7), rng.normal(size=(4, 7))
    y, r = on.forward(np.full((1, 5), 3.0), np.arange(5.0), 0.0)
    assert np.allclose(y, np.arange(5.0)) and np.allclose(r, 1 / 3)
    y, r = on.forward(h, w, 1e-3)
    d, dw = on.backward(dy, h, w, r)
    step = 1e-6
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = step
        up, down = (on.forward(h + s * e, w, 1e-3)[0] for s in (1, -1))
        assert abs(np.sum((up - down) * dy) / (2 * step) - d[i]) <= 1e-8
    for i in range(7):
        e = np.zeros(7)
        e[i] = step
        up, down = (on.forward(h, w + s * e, 1e-3)[0] for s in (1, -1))
        assert abs(np.sum((up - down) * dy) / (2 * step) - dw[i]) <= 1e-8


def test_row_scale():
    y = np.array([[448.0, 1.0], [448.1, 0.0], [0.0, 0.0], [1.75, -1.0], [-3.6, 0.0], [1e-44, 0.0]])
    assert on.row_scale(y).tolist() == [1.0, 2.0, 1.0, 2.0 ** -8, 2.0 ** -6, 2.0 ** -126]


def drop(p=0.1, seed=1, offset=0, state=None):
    return _lib.Dropout(p=p, seed=seed, offset=offset, state=state)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(d=None), BAD), (dict(dt=2), BAD),
    (dict(d=drop(-0.1)), BAD), (dict(d=drop(1.0)), BAD), (dict(d=drop(math.nan)), BAD),
    (dict(d=drop(1 - 2.0 ** -40)), BAD), (dict(d=drop(state=FAKE + 4)), BAD),
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(x=FAKE + 1), BAD), (dict(y=FAKE + 2, dt=1), BAD),
    (dict(ys=63), BAD), (dict(ys=0), BAD), (dict(y=FAKE, ys=128), BAD),
    (dict(cols=1 << 31), UNSUP), (dict(rows=1 << 37, cols=1), UNSUP), (dict(rows=1 << 34, cols=128), UNSUP),
])
def test_dropout_rejects(kw, code):
    a = dict(x=FAKE, rows=10, cols=64, xs=64, ys=64, d=drop(), dt=0, y=2 * FAKE)
    a.update(kw)
    d = None if a["d"] is None else ctypes.byref(a["d"])
    assert L.lora_dropout(a["x"], a["rows"], a["cols"], a["xs"], a["ys"], d, a["dt"], a["y"], None) == code
    assert L.lora_last_error().decode() != ""


def test_dropout_nothing_to_do():
    d = drop()
    for rows, cols in ((0, 5), (5, 0)):
        assert L.lora_dropout(None, rows, cols, 0, 0, ctypes.byref(d), 0, None, None) == _lib.LORA_OK


def norm_shape(**kw):
    a = dict(outer=10, inner=1, dim=64, weight_fp32=0, eps=1e-6)
    a.update({n: (64, 0) for n in ("x", "residual", "h", "y", "dy", "dh", "dx", "dresidual")})
    a.update(kw)
    return _lib.NormShape(**a)


def norm_fwd(ptr, **kw):
    a = dict(x=FAKE, residual=2 * FAKE, w=3 * FAKE, d=None, dt=0, h=4 * FAKE, y=5 * FAKE, rstd=6 * FAKE,
             codes=None, scale=None)
    a.update(ptr)
    d = None if a["d"] is None else ctypes.byref(a["d"])
    return L.lora_norm_fwd(ctypes.byref(norm_shape(**kw)), a["x"], a["residual"], a["w"], d, a["dt"],
                           a["h"], a["y"], a["rstd"], a["codes"], a["scale"], None)


def norm_bwd(ptr, **kw):
    a = dict(dy=FAKE, h=2 * FAKE, w=3 * FAKE, rstd=4 * FAKE, dh=5 * FAKE, d=None, dt=0, dx=6 * FAKE,
             dres=None, dw=7 * FAKE, ws=8 * FAKE, n=1 << 20)
    a.update(ptr)
    d = None if a["d"] is None else ctypes.byref(a["d"])
    return L.lora_norm_bwd(ctypes.byref(norm_shape(**kw)), a["dy"], a["h"], a["w"], a["rstd"], a["dh"], d,
                           a["dt"], a["dx"], a["dres"], a["dw"], a["ws"], a["n"], None)


BAD_SHAPES = [(dict(outer=-1), BAD), (dict(inner=-1), BAD), (dict(dim=0), BAD), (dict(dim=32769), UNSUP),
              (dict(weight_fp32=2), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
              (dict(eps=math.inf), BAD), (dict(outer=1 << 20, inner=1 << 11), UNSUP),
              (dict(outer=1 << 62, inner=4), UNSUP), (dict(outer=0, inner=1 << 40), UNSUP)]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_norm_rejects_shapes(kw, code):
    assert norm_fwd({}, **kw) == code
    assert L.lora_last_error().decode() != ""
    assert norm_bwd({}, **kw) == code
    assert L.lora_last_error().decode() != ""


@pytest.mark.parametrize("ptr,kw", [
    (dict(x=None), {}), (dict(w=None), {}), (dict(x=FAKE + 1), {}), (dict(y=FAKE + 2, dt=1), {}),
    (dict(w=FAKE + 2), dict(weight_fp32=1)), (dict(rstd=FAKE + 2), {}), (dict(codes=FAKE), {}),
    (dict(scale=FAKE), {}), (dict(dt=3), {}), (dict(d=drop(2.0)), {}),
    (dict(residual=None), {}),                       # h given, but it is x
    (dict(y=None, h=None), {}),                      # nothing to write
    (dict(y=4 * FAKE), {}),                          # y is h
    ({}, dict(y=(63, 0))), ({}, dict(h=(0, 0))), ({}, dict(outer=2, inner=5, y=(640, 32))),
    (dict(h=2 * FAKE), dict(h=(128, 0))),            # in place with other strides
    (dict(y=FAKE), dict(y=(128, 0))),
])
def test_norm_forward_rejects(ptr, kw):
    assert norm_fwd(ptr, **kw) == BAD
    assert L.lora_last_error().decode() != ""


@pytest.mark.parametrize("ptr,kw,code", [
    (dict(dy=None), {}, BAD), (dict(h=None), {}, BAD), (dict(w=None), {}, BAD), (dict(rstd=None), {}, BAD),
    (dict(dx=None), {}, BAD), (dict(dx=FAKE + 1), {}, BAD), (dict(dres=6 * FAKE), {}, BAD),
    (dict(dw=FAKE + 2), dict(weight_fp32=1), BAD), (dict(rstd=FAKE + 2), {}, BAD),
    (dict(dx=FAKE), dict(dx=(128, 0)), BAD), ({}, dict(dx=(0, 0)), BAD), (dict(d=drop(-1.0)), {}, BAD),
    (dict(ws=None), {}, WS), (dict(n=64 * 4 - 1), {}, WS), (dict(ws=FAKE + 8), {}, BAD),
])
def test_norm_backward_rejects(ptr, kw, code):
    assert norm_bwd(ptr, **kw) == code
    assert L.lora_last_error().decode() != ""


def test_norm_nothing_to_do():
    assert norm_fwd(dict(x=None, residual=None, h=None, y=None, w=None), outer=0) == _lib.LORA_OK
    assert norm_bwd(dict(dy=None, h=None, w=None, rstd=None, dx=None, dw=None), outer=0) == _lib.LORA_OK


def test_norm_workspace():
    assert L.lora_norm_workspace_bytes(ctypes.byref(norm_shape(outer=3, dim=4096)), 1) == 3 * 4096 * 4
    assert L.lora_norm_workspace_bytes(ctypes.byref(norm_shape()), 0) == 0
    assert L.lora_norm_workspace_bytes(ctypes.byref(norm_shape(dim=0)), 1) == 0


def test_fp8_rows_rejects():
    def call(**kw):
        a = dict(X=FAKE, Xq=2 * FAKE, xs=3 * FAKE, r=16)
        a.update(kw)
        return L.lora_fp8_fwd_rows(a["X"], a["Xq"], a["xs"], FAKE, FAKE, FAKE, FAKE, 1.0, a["r"], 32, 64, 64,
                                   FAKE, FAKE, FAKE, 1 << 30, None)
    for kw in (dict(X=None), dict(Xq=None), dict(Xq=FAKE + 8), dict(xs=None), dict(xs=FAKE + 2), dict(r=0)):
        assert call(**kw) != _lib.LORA_OK
        assert L.lora_last_error().decode() != ""


def test_python_refuses_what_is_not_on_a_gpu():
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises((ValueError, TypeError)):
        rl.rms_norm_forward(x, w)
    with pytest.raises((ValueError, TypeError)):
        rl.dropout_forward(x, 0.1, 1)
    with pytest.raises(ValueError):
        rl.dropout(torch.zeros(()), 0.1, 1)
