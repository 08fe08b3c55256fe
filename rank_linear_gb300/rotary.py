"""Rotary positions of q and k (ch05 "Acceleration principles: Triton kernels
and fused LoRA", §5.5): what stands between the q and k LoRA layers and the
attention.  Both tensors are turned in one launch of the CUDA library; angles
are as good at position 2^41 as at 1 (see include/lora_rotary.h).
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .lora import _dtype_code, _ptr


class RotaryFrequencies:
    """Frequencies of a head's rotated pairs, on the device: what a program
    keeps beside its weights.  `radians` are the frequencies per position,
    `magnitude` the factor on the rotated elements."""

    def __init__(self, radians, magnitude: float = 1.0, device=None):
        self.radians = [float(w) for w in radians]
        self.magnitude = float(magnitude)
        n = len(self.radians)
        words = (ctypes.c_uint64 * max(n, 1))()
        _lib.check(_lib.lib().lora_rotary_turns((ctypes.c_double * max(n, 1))(*self.radians), n,
                                                words), "lora_rotary_turns")
        signed = [w - (1 << 64) if w >> 63 else w for w in words[:n]]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.device = self.turns.device
        self.rot = 2 * n


def rotary_frequencies(rot: int, *, base: float = 10000.0, scaling: dict | None = None,
                       device=None) -> RotaryFrequencies:
    """w_i = base^(-2i / rot), i < rot / 2, scaled for long contexts by `scaling`:

    None
        as they are.
    {"kind": "linear", "factor": f}
        every frequency divided by f (positions squeezed into the trained range).
    {"kind": "base", "factor": f}
        the base times f^(rot / (rot - 2)): the slowest pair is stretched f
        times, the fastest not at all.
    {"kind": "bands", "factor": f, "original": n, "low": a, "high": b}
        by the turns t a pair makes over the n trained positions: kept for
        t >= b, divided by f for t <= a, between them the blend
        (t - a) / (b - a) of the two frequencies.
    {"kind": "ramp", "factor": f, "original": n, "fast": a, "slow": b}
        the same blend along a linear ramp over the pair's index, from the
        pair that makes a turns over n positions (kept) to the one that makes
        b; rotated elements are scaled by 0.1 ln f + 1, or by "magnitude".
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot = {rot} is not an even number >= 2")
    if not (base > 0 and math.isfinite(base)):
        raise ValueError(f"base = {base}")
    s = dict(scaling or {})
    kind = s.pop("kind", None)
    need = {None: (), "linear": ("factor",), "base": ("factor",),
            "bands": ("factor", "original", "low", "high"),
            "ramp": ("factor", "original", "fast", "slow")}
    if kind not in need:
        raise ValueError(f"scaling kind {kind!r} is not one of {sorted(k for k in need if k)}")
    magnitude = float(s.pop("magnitude", 0.1 * math.log(s.get("factor", 1.0)) + 1.0)) \
        if kind == "ramp" else 1.0
    if sorted(s) != sorted(need[kind]):
        raise ValueError(f"scaling {kind!r} takes {need[kind]}, got {sorted(s)}")
    for name, value in s.items():
        if not (value > 0 and math.isfinite(value)):
            raise ValueError(f"scaling {name} = {value} must be positive")
    f = s.get("factor", 1.0)
    if kind == "base" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        w = [x / f for x in w]
    elif kind == "bands":
        if not s["high"] > s["low"]:
            raise ValueError("scaling 'bands' needs high > low")

        def band(x):
            keep = (s["original"] * x / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])
            keep = min(1.0, max(0.0, keep))
            return keep * x + (1.0 - keep) * x / f
        w = [band(x) for x in w]
    elif kind == "ramp":
        def pair_of(turns):  # index of the pair that makes so many turns over `original`
            return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair_of(s["fast"])), 0)
        hi = min(math.ceil(pair_of(s["slow"])), rot - 1)
        go = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        w = [(1.0 - g) * x + g * x / f for x, g in zip(w, go)]
    return RotaryFrequencies(w, magnitude, device)


def _strides(t, name, device):
    """(batch, token, head) strides of [batch, seq, heads, dim] or [tokens, heads, dim]."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _same_device(t, name, device)
    if t.dim() == 4:
        s = t.stride()
    elif t.dim() == 3:
        s = (0,) + t.stride()
    else:
        raise ValueError(f"{name} must be [batch, seq, heads, dim] or [tokens, heads, dim]")
    if s[3] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return s[:3]


def _empty_like(t):
    # (a third of the time of torch.empty with a shape, a type and a device)
    return torch.empty_like(t, memory_format=torch.contiguous_format)


_here = contextlib.nullcontext()


def _on(stream):
    """Buffers made for work on another stream come from that stream's pool."""
    return _here if stream is None else torch.cuda.stream(stream)


def _same_device(t, name, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _stream_on(device, stream):
    """The handle to launch on: the current stream's where none is given.  The
    library launches on the current device, which has to be the tensors'."""
    at = torch.cuda.current_device()
    if at != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{at}")
    if stream is None:  # without making an object of it
        return torch._C._cuda_getCurrentRawStream(at) or None
    return stream.cuda_stream or None


def _layout(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


# Argument blocks by the layouts that they describe (sizes, strides, types;
# no addresses): checking and filling one takes longer than a small launch.
_blocks: dict = {}
_MOST_BLOCKS = 4096


def _block(key, make):
    block = _blocks.get(key)
    if block is None:
        block = make()
        if len(_blocks) >= _MOST_BLOCKS:
            _blocks.clear()
        _blocks[key] = block
    return block


def _make_shape(q, k, positions, freqs, interleaved, inverse, q_out, k_out):
    first = q if q is not None else k
    sh = _lib.RotaryShape()
    lead = first.shape[:-2]
    if len(lead) not in (1, 2):
        raise ValueError("q and k must be [batch, seq, heads, dim] or [tokens, heads, dim]")
    sh.batch, sh.seq = (1, lead[0]) if len(lead) == 1 else lead
    sh.dim, sh.rot = first.shape[-1], freqs.rot
    sh.interleaved, sh.inverse, sh.magnitude = int(interleaved), int(inverse), freqs.magnitude
    for name, x, out in (("q", q, q_out), ("k", k, k_out)):
        if x is None:
            continue
        if x.shape[:-2] != lead or x.shape[-1] != first.shape[-1] or out.shape != x.shape:
            raise ValueError(f"{name} {tuple(x.shape)} and its output {tuple(out.shape)} do not fit")
        if x.dtype != first.dtype or out.dtype != first.dtype:
            raise TypeError("q, k and the outputs must share one dtype")
        setattr(sh, name + "_heads", x.shape[-2])
        setattr(sh, name + "_in", _strides(x, name, first.device))
        setattr(sh, name + "_out", _strides(out, name + "_out", first.device))
    if positions.dtype not in (torch.int32, torch.int64) or not positions.is_cuda:
        raise TypeError("positions must be an int32 or int64 CUDA tensor")
    _same_device(positions, "positions", first.device)
    sh.position_bits = 64 if positions.dtype == torch.int64 else 32
    if positions.shape == lead:
        sh.position = positions.stride() if len(lead) == 2 else (0, positions.stride(0))
    elif len(lead) == 2 and positions.shape == lead[1:]:
        sh.position = (0, positions.stride(0))
    else:
        raise ValueError(f"positions {tuple(positions.shape)} do not fit tokens {tuple(lead)}")
    if freqs.device != first.device:
        raise ValueError("the frequencies are on another device")
    return sh, _dtype_code(first)


def _turn(q, k, positions, freqs, interleaved, inverse, q_out, k_out, stream):
    if q is None and k is None:
        raise ValueError("q and k are both None")
    # (an output made here has the layout that its input's decides)
    interleaved, magnitude = bool(interleaved), float(freqs.magnitude)  # a tensor's: as it is now
    key = (_layout(q), _layout(k), _layout(positions), _layout(q_out), _layout(k_out),
           freqs.rot, magnitude, freqs.device, interleaved, inverse)
    if q_out is None or k_out is None:
        with _on(stream):
            if q is not None and q_out is None:
                q_out = _empty_like(q)
            if k is not None and k_out is None:
                k_out = _empty_like(k)
    sh, dtype = _block(key, lambda: _make_shape(q, k, positions, freqs, interleaved, inverse,
                                                q_out, k_out))
    st = _lib.lib().lora_rotary(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(positions),
                                _ptr(freqs.turns), dtype, _ptr(q_out), _ptr(k_out),
                                _stream_on((k if q is None else q).device, stream))
    if st:
        _lib.check(st, "lora_rotary")
    return q_out, k_out


def rotary_forward(q, k, positions, freqs: RotaryFrequencies, *, interleaved=False, q_out=None,
                   k_out=None, stream=None):
    """(q, k) turned by their tokens' positions; q or k may be None.

    q and k are [batch, seq, heads, dim] or [tokens, heads, dim], the elements of
    a head side by side, with any other strides (views of a fused q|k|v output); positions [batch, seq], [seq] or
    [tokens].  q_out / k_out may be q / k themselves (in place)."""
    return _turn(q, k, positions, freqs, interleaved, False, q_out, k_out, stream)


def rotary_backward(dq, dk, positions, freqs: RotaryFrequencies, *, interleaved=False,
                    dq_out=None, dk_out=None, stream=None):
    """Gradients of the inputs from those of rotary_forward's outputs."""
    return _turn(dq, dk, positions, freqs, interleaved, True, dq_out, dk_out, stream)


def _fit(t):
    """t itself where a head's elements lie side by side, else a copy."""
    return t if t is None or t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class RotaryFunction(torch.autograd.Function):
    """Autograd function: saves the positions only.  Gradients once (not gradients
    of gradients)."""

    @staticmethod
    def forward(ctx, q, k, positions, freqs, interleaved):
        ctx.save_for_backward(positions)
        ctx.freqs, ctx.interleaved = freqs, interleaved
        return rotary_forward(_fit(q), _fit(k), positions, freqs, interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        positions, = ctx.saved_tensors
        dq, dk = rotary_backward(_fit(dq), _fit(dk), positions, ctx.freqs,
                                 interleaved=ctx.interleaved)
        return dq, dk, None, None, None


def rotary(q, k, positions, freqs: RotaryFrequencies, *, interleaved=False):
    """Rotary positions of q and k (with any strides) with gradients for both."""
    return RotaryFunction.apply(q, k, positions, freqs, interleaved)
