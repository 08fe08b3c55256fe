"""The loss's oracle against closed forms and differences, and the refusals of the
entry points, on the CPU (no launches)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rank_linear_gb300 as rl
from oracle import head_loss as ol
from rank_linear_gb300 import _lib, build

FAKE = 0x100000  # aligned non-null "device" address; never dereferenced here
BAD, UNSUP, WS = _lib.LORA_ERR_INVALID_ARG, _lib.LORA_ERR_UNSUPPORTED, _lib.LORA_ERR_WORKSPACE
L = None


def setup_module():
    global L
    build.build()
    L = _lib.lib()


def test_closed_forms():
    x, w = np.zeros((3, 8)), np.ones((10, 8))
    r = ol.run(x, w, np.array([0, 9, -1]))
    assert np.allclose(r["losses"], [math.log(10), math.log(10), 0]) and abs(r["loss"] - math.log(10)) < 1e-12
    # two words: the logistic loss
    x, w = np.array([[2.0]]), np.array([[1.0], [-0.5]])
    for t, d in ((0, 3.0), (1, -3.0)):
        r = ol.run(x, w, np.array([t]))
        p = 1 / (1 + math.exp(-d))
        assert abs(r["loss"] - math.log1p(math.exp(-d))) < 1e-12
        assert abs(r["dx"][0, 0] - (1 - p) * (w[1 - t] - w[t])[0]) < 1e-12
    # hopeless and certain targets
    x = np.array([[400.0]])
    assert abs(ol.run(x, w, np.array([1]))["loss"] - 600) < 1e-9
    assert ol.run(x, w, np.array([0]))["loss"] == math.exp(-600)


@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_gradient_is_the_differences(cap):
    rng = np.random.default_rng(3)
    x, w = rng.normal(size=(5, 4)), rng.normal(size=(9, 4))
    t, g = np.array([3, -1, 0, 8, 3]), rng.random(5)
    r = ol.run(x, w, t, g, cap)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-6
        up, down = (ol.run(x + s * e, w, t, g, cap)["loss"] for s in (1, -1))
        assert abs((up - down) / 2e-6 - r["dx"][i]) < 1e-8


def shape(**kw):
    a = dict(rows=10, vocab=100, dim=64, target_bits=64, mean=1, softcap=0.0, x=64, w=64, dx=64)
    a.update(kw)
    return _lib.LossShape(**a)


def call(ptr=None, **kw):
    a = dict(X=FAKE, W=2 * FAKE, t=3 * FAKE, w=4 * FAKE, loss=5 * FAKE, each=6 * FAKE, dX=7 * FAKE,
             ws=8 * FAKE, n=1 << 40)
    a.update(ptr or {})
    return L.lora_loss(ctypes.byref(shape(**kw)), a["X"], a["W"], a["t"], a["w"], a["loss"], a["each"],
                       a["dX"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), BAD), (dict(vocab=0), BAD), (dict(dim=0), BAD), (dict(dim=60), UNSUP),
    (dict(dim=65544, x=65544, w=65544, dx=65544), UNSUP), (dict(rows=2 ** 31 - 65536), UNSUP),
    (dict(vocab=2 ** 31 - 511), UNSUP), (dict(target_bits=16), BAD), (dict(mean=2), BAD),
    (dict(softcap=-1.0), BAD), (dict(softcap=math.inf), BAD), (dict(softcap=math.nan), BAD),
    (dict(x=60), BAD), (dict(x=68), BAD), (dict(w=0), BAD), (dict(dx=56), BAD),
])
def test_rejects_shapes(kw, code):
    assert call(**kw) == code
    assert L.lora_last_error().decode() != ""


@pytest.mark.parametrize("ptr,kw,code", [
    (dict(X=None), {}, BAD), (dict(W=None), {}, BAD), (dict(t=None), {}, BAD), (dict(loss=None), {}, BAD),
    (dict(each=None), {}, BAD), (dict(X=FAKE + 8), {}, BAD), (dict(W=FAKE + 8), {}, BAD),
    (dict(dX=FAKE + 8), {}, BAD), (dict(t=FAKE + 4), {}, BAD), (dict(w=FAKE + 2), {}, BAD),
    (dict(loss=FAKE + 2), {}, BAD), (dict(each=FAKE + 2), {}, BAD), (dict(dX=2 * FAKE), {}, BAD),
    (dict(dX=FAKE), dict(dx=128), BAD), (dict(ws=None), {}, WS), (dict(n=1000), {}, WS),
    (dict(ws=FAKE + 8), {}, BAD),
])
def test_rejects(ptr, kw, code):
    assert call(ptr, **kw) == code
    assert L.lora_last_error().decode() != ""


def test_workspace_is_bounded():
    """A strip's exponentials and sums, not the logits of all tokens."""
    need = lambda grad, **kw: L.lora_loss_workspace_bytes(ctypes.byref(shape(**kw)), grad)
    big = dict(vocab=128000, dim=4096, x=4096, w=4096, dx=4096)
    assert need(1, rows=8192, **big) < 0.75e9 and need(1, rows=65536, **big) < 0.75e9
    assert need(0, rows=65536, **big) < 0.7e9
    assert need(0, rows=8, **big) < need(1, rows=8, **big)
    assert need(1, dim=60) == 0


def test_scale_rejects():
    call = lambda dX=FAKE, f=FAKE, out=2 * FAKE, **kw: L.lora_loss_scale(ctypes.byref(shape(**kw)), dX, f,
                                                                         out, None)
    for kw in (dict(dX=None), dict(out=None), dict(f=None), dict(f=FAKE + 2), dict(out=FAKE, x=128),
               dict(x=8), dict(dim=3)):
        assert call(**kw) != _lib.LORA_OK
        assert L.lora_last_error().decode() != ""
    assert call(rows=0, dX=None, out=None, f=None) == _lib.LORA_OK


def test_python_refusals():
    x, w = torch.zeros(4, 8).bfloat16(), torch.zeros(5, 8).bfloat16()
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises((TypeError, ValueError)):
        rl.cross_entropy_forward(x, w, t)
    with pytest.raises(ValueError):
        rl.cross_entropy_forward(x, w, t, reduction="none")


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("rows", [1, 300, 8192, 65536, 1 << 20])
@pytest.mark.parametrize("vocab,dim", [(1, 8), (100, 64), (1000, 65536), (4096, 5120), (8192, 8192), (32000, 4096),
                                       (128000, 4096), (128000, 65536), (2_000_003, 64), (2 ** 31 - 512, 8)])
def test_workspace_bound_of_any_shape(vocab, dim, rows, grad):
    """716 MB (of 2^20) and four bytes a token; or where 256 tokens take more than 640 of them, what
    these take: two bytes a word and element of X, eight a piece of 128 words (of whole tiles of 512), and
    numbers of their own; and 76 MB of partial tiles."""
    need = L.lora_loss_workspace_bytes(ctypes.byref(shape(rows=rows, vocab=vocab, dim=dim)), grad)
    least = 256 * (2 * (vocab + 7) + 2 * dim + 8 * ((vocab + 511) // 512 * 4) + 16)
    assert 0 < need <= max(640 << 20, least) + (76 << 20) + 4 * rows + 4096
