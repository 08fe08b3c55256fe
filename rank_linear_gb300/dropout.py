"""Dropout whose mask is made again from (seed, offset) instead of stored
(include/lora_dropout.h; the Unsloth essay's recipe table names the rate)."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .lora import _dtype_code, _ptr
from .rotary import _block, _empty_like, _layout, _on, _same_device, _stream_on


def _seed_of(seed, device):
    """(layout key, seed word, state tensor): a number, or an int64 tensor of two words
    (seed, offset) on the device, which is read when the kernel runs."""
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.shape != (2,) or not seed.is_contiguous() or not seed.is_cuda:
            raise ValueError("seed must be a number or a contiguous int64 CUDA tensor of (seed, offset)")
        _same_device(seed, "seed", device)
        return 0, seed
    seed = int(seed)
    if not -2 ** 63 <= seed < 2 ** 64:
        raise ValueError(f"seed = {seed} does not fit 64 bits")
    return seed % 2 ** 64, None


_KEEP = _lib.Dropout()  # p = 0


def _drop_block(p, seed, offset, device):
    """The dropout's argument block (None: no dropout) and what keeps its address alive."""
    p = float(p)
    if p == 0.0:
        return None
    offset = int(offset)
    if not 0 <= offset < 2 ** 32:
        raise ValueError(f"offset = {offset} does not fit 32 bits")
    word, state = _seed_of(seed, device)
    return _lib.Dropout(p, word, offset, _ptr(state))


def _collapsed(shape, strides):
    """The one stride of these dimensions taken as one (0 for a single entry), or None."""
    step, size = None, 1
    for n, s in zip(reversed(shape), reversed(strides)):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != step * size:
            return None
        size *= n
    return step or 0


def _check(t, name, like):
    if t.dim() < 1:
        raise ValueError(f"{name} has no dimension")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _same_device(t, name, like.device)
    if t.shape != like.shape:
        raise ValueError(f"{name} {tuple(t.shape)} is not {tuple(like.shape)}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} is {t.dtype}, not {like.dtype}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")


def _make(x, out):
    _check(x, "x", x)
    _check(out, "out", x)
    steps = [_collapsed(t.shape[:-1], t.stride()[:-1]) for t in (x, out)]
    if None in steps:
        raise ValueError("the rows of x and out must lie one stride apart")
    cols = x.shape[-1]
    return (x.numel() // cols if cols else 0, cols, *steps), _dtype_code(x)


def dropout_forward(x, p, seed, offset=0, *, out=None, stream=None):
    """x [..., columns] with each element kept with probability 1 - p and then
    divided by it, else 0.

    p        0 <= p < 1, as a multiple of 2^-32.
    seed     a number of 64 bits, or an int64 CUDA tensor (seed, offset) that is
             read when the kernel runs (for captured graphs; its offset is added).
    offset   32 bits: another mask of the same seed for each use in a step.
    out      may be x itself (in place).
    """
    # (an output made here has the layout that x's decides)
    key = ("dropout", _layout(x), _layout(out))
    if out is None:
        if stream is None:
            out = _empty_like(x)
        else:
            with _on(stream):
                out = _empty_like(x)
    (rows, cols, xs, ys), dtype = _block(key, lambda: _make(x, out))
    block = _drop_block(p, seed, offset, x.device) or _KEEP
    st = _lib.lib().lora_dropout(_ptr(x), rows, cols, xs, ys, ctypes.byref(block), dtype, _ptr(out),
                                 _stream_on(x.device, stream))
    if st:
        _lib.check(st, "lora_dropout")
    return out


def dropout_backward(dout, p, seed, offset=0, *, out=None, stream=None):
    """The gradient of dropout_forward's x from that of its output."""
    return dropout_forward(dout, p, seed, offset, out=out, stream=stream)


def _fit(t):
    """t itself where its rows suit the kernels, else a contiguous copy."""
    ok = (t.shape[-1] <= 1 or t.stride(-1) == 1) and \
        _collapsed(t.shape[:-1], t.stride()[:-1]) is not None
    return t if ok else t.contiguous()


def _kept_seed(seed):
    """A tensor's words as they are now, for the backward."""
    return seed.clone() if isinstance(seed, torch.Tensor) else seed


class DropoutFunction(torch.autograd.Function):
    """Autograd function: saves the seed only.  Gradients once (not gradients of
    gradients)."""

    @staticmethod
    def forward(ctx, x, p, seed, offset):
        # (the backward's are the forward's, whatever a tensor of them holds then)
        ctx.args = (float(p), _kept_seed(seed), int(offset))
        return dropout_forward(_fit(x), *ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        return dropout_backward(_fit(dout), *ctx.args), None, None, None


def dropout(x, p, seed, offset=0):
    """dropout_forward's output with the gradient of x (of any strides)."""
    if x.dim() < 1:
        raise ValueError("x has no dimension")
    return DropoutFunction.apply(x, p, seed, offset)
