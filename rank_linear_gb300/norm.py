"""Root-mean-square norm with the residual's addition, dropout of the branch and
an 8-bit output for the fp8 layers (formulas in include/lora_norm.h; ch05
"Acceleration principles: Triton kernels and fused LoRA", §5.4)."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .dropout import _check, _collapsed, _drop_block, _kept_seed
from .lora import _dtype_code, _ptr
from .rotary import _block, _empty_like, _layout, _on, _same_device, _stream_on


def _row_strides(tensors):
    """(outer, inner, [(outer stride, inner stride)]) of tensors of one shape: their
    leading dimensions as two, the second 1 where every tensor's are one; None
    where no split suits them all."""
    lead = tensors[0].shape[:-1]
    for at in range(len(lead), -1, -1):
        strides = []
        for t in tensors:
            a, b = _collapsed(lead[:at], t.stride()[:at]), _collapsed(lead[at:], t.stride()[at:-1])
            if a is None or b is None:
                break
            strides.append((a, b))
        else:
            return lead[:at].numel(), lead[at:].numel(), strides
    return None


def _check_weight(weight, x, name="weight"):
    if weight.shape != x.shape[-1:] or not weight.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {x.shape[-1]} elements")
    if weight.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"{name} is {weight.dtype}, not {x.dtype} or float32")
    _same_device(weight, name, x.device)


def _make(first, weight, eps, tensors):
    """The argument block without addresses; tensors: by their names in it."""
    for name, t in tensors.items():
        _check(t, name, first)
    _check_weight(weight, first)
    dtype = _dtype_code(first)
    split = _row_strides(list(tensors.values()))
    if split is None:
        raise ValueError("the rows of these tensors do not lie on two common strides")
    outer, inner, strides = split
    sh = _lib.NormShape(outer=outer, inner=inner, dim=first.shape[-1], eps=eps,
                        weight_fp32=int(weight.dtype == torch.float32))
    for name, s in zip(tensors, strides):
        setattr(sh, name, s)
    return sh, dtype


def _row_floats(t, name, like):
    if t.dtype != torch.float32 or not t.is_contiguous() or t.shape != like.shape[:-1] or \
            t.device != like.device:
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(like.shape[:-1])}")


def _outputs(x, out, h_out, summed, fp8):
    if out is None:
        out = _empty_like(x)
    if h_out is None and summed:
        h_out = _empty_like(x)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    if not fp8:
        return out, h_out, rstd, None, None
    return out, h_out, rstd, torch.empty(x.shape, dtype=torch.uint8, device=x.device), torch.empty_like(rstd)


def rms_norm_forward(x, weight, *, residual=None, eps=1e-6, dropout=0.0, seed=0, offset=0,
                     fp8=False, out=None, h_out=None, stream=None):
    """(y, h, rstd) of x [..., dim]: h = dropout(x) + residual, y = h * rstd * weight
    with rstd = (mean of h^2 + eps)^-1/2 of each row (float32 [...]).

    weight    [dim], of x's type or float32.
    residual  like x, or None.  Without it and dropout, h is x itself.
    dropout   probability; seed and offset as dropout_forward's.
    fp8       also returns (codes [..., dim] uint8, scale [...] float32): y in e4m3
              with a power of two for each row, as fp8_forward takes them (rows=).
    out       may be x (without residual and dropout the h returned is then y, and the input
              is gone); h_out may be residual (the stream updated in place) or x.
    """
    drop = _drop_block(dropout, seed, offset, x.device)
    eps, summed = float(eps), residual is not None or drop is not None
    if h_out is not None and not summed:
        raise ValueError("h is x without residual and dropout")
    # (outputs made here have the layouts that x's decides)
    key = ("norm", _layout(x), _layout(weight), _layout(residual), _layout(out), _layout(h_out), summed, eps)
    if stream is None:
        out, h_out, rstd, codes, scale = _outputs(x, out, h_out, summed, fp8)
    else:
        with _on(stream):
            out, h_out, rstd, codes, scale = _outputs(x, out, h_out, summed, fp8)

    def make():
        given = {"x": x, "residual": residual, "h": h_out, "y": out}
        return _make(x, weight, eps, {n: t for n, t in given.items() if t is not None})
    sh, dtype = _block(key, make)
    st = _lib.lib().lora_norm_fwd(ctypes.byref(sh), _ptr(x), _ptr(residual), _ptr(weight),
                                  None if drop is None else ctypes.byref(drop), dtype, _ptr(h_out),
                                  _ptr(out), _ptr(rstd), _ptr(codes), _ptr(scale),
                                  _stream_on(x.device, stream))
    if st:
        _lib.check(st, "lora_norm_fwd")
    h = h_out if summed else x
    return (out, h, rstd, codes, scale) if fp8 else (out, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, *, dh=None, dropout=0.0, seed=0, offset=0,
                      need_dweight=True, dx=None, dresidual=None, dweight=None, workspace=None,
                      stream=None):
    """(dx, dresidual, dweight or None) from the gradient dy of rms_norm_forward's y and
    the gradient dh that reaches its h otherwise (None: 0).  Without dropout,
    dresidual is dx.  dx or dresidual may be dy or dh (in place)."""
    drop = _drop_block(dropout, seed, offset, dy.device)
    if drop is None and dresidual is not None:
        raise ValueError("without dropout dresidual is dx")
    # (gradients made here have the layouts that dy's decides)
    key = ("norm backward", _layout(dy), _layout(h), _layout(weight), _layout(rstd), _layout(dh),
           _layout(dx), _layout(dresidual), _layout(dweight), drop is None, need_dweight)

    def buffers():
        return (_empty_like(dy) if dx is None else dx,
                _empty_like(dy) if dresidual is None and drop is not None else dresidual,
                torch.empty_like(weight) if need_dweight and dweight is None else dweight)

    def make():
        given = {"dy": dy, "h": h, "dh": dh, "dx": dx, "dresidual": dresidual}
        sh, dtype = _make(dy, weight, 0.0, {n: t for n, t in given.items() if t is not None})
        _row_floats(rstd, "rstd", dy)
        if need_dweight:
            _check_weight(dweight, dy, "dweight")
            if dweight.dtype != weight.dtype:
                raise TypeError(f"dweight is {dweight.dtype}, not {weight.dtype}")
        return sh, dtype, _lib.lib().lora_norm_workspace_bytes(ctypes.byref(sh), int(need_dweight))

    def scratch():
        return torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    if workspace is not None and (workspace.device != dy.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the device of dy")
    if stream is None:
        dx, dresidual, dweight = buffers()
        sh, dtype, need = _block(key, make)
        workspace = scratch() if workspace is None else workspace
    else:
        with _on(stream):
            dx, dresidual, dweight = buffers()
            sh, dtype, need = _block(key, make)
            workspace = scratch() if workspace is None else workspace
    st = _lib.lib().lora_norm_bwd(ctypes.byref(sh), _ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd),
                                  _ptr(dh), None if drop is None else ctypes.byref(drop), dtype,
                                  _ptr(dx), _ptr(dresidual), _ptr(dweight) if need_dweight else None,
                                  _ptr(workspace),
                                  0 if workspace is None else workspace.numel() * workspace.element_size(),
                                  _stream_on(dy.device, stream))
    if st:
        _lib.check(st, "lora_norm_bwd")
    return dx, (dx if drop is None else dresidual), (dweight if need_dweight else None)


def _fit_rows(*tensors):
    """The tensors themselves where their rows suit the kernels together, else
    contiguous copies of those given."""
    given = [t for t in tensors if t is not None]
    if all(t.shape[-1] <= 1 or t.stride(-1) == 1 for t in given) and _row_strides(given) is not None:
        return tensors
    return tuple(None if t is None else t.contiguous() for t in tensors)


class RMSNormFunction(torch.autograd.Function):
    """Autograd function: saves h, the weight and rstd.  Gradients for x, the weight and
    the residual, once (not gradients of gradients)."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, dropout, seed, offset, fp8):
        ctx.set_materialize_grads(False)
        x, residual = _fit_rows(x, residual)
        weight = weight.contiguous()
        ctx.drop = dict(dropout=float(dropout), seed=_kept_seed(seed), offset=int(offset))
        ctx.has_residual = residual is not None
        y, h, rstd, *rows = rms_norm_forward(x, weight, residual=residual, eps=eps, fp8=fp8, **ctx.drop)
        ctx.save_for_backward(h, weight, rstd)
        out = (y,) + ((h,) if ctx.has_residual else ()) + tuple(rows)
        if rows:
            ctx.mark_non_differentiable(*rows)
        return out if len(out) > 1 else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, *rest):
        h, weight, rstd = ctx.saved_tensors
        dh = rest[0] if ctx.has_residual else None
        if dy is None and dh is None:
            return (None,) * 8
        dy, h, dh = _fit_rows(torch.zeros_like(h) if dy is None else dy, h, dh)
        dx, dres, dw = rms_norm_backward(dy, h, weight, rstd, dh=dh, need_dweight=ctx.needs_input_grad[1],
                                         **ctx.drop)
        return dx, dw, (dres if ctx.has_residual else None), None, None, None, None, None


def rms_norm(x, weight, *, residual=None, eps=1e-6, dropout=0.0, seed=0, offset=0, fp8=False):
    """rms_norm_forward's y with gradients for x, weight and residual: y, or (y, h) with
    a residual (h: the stream that goes on), and the codes and scale after them
    with fp8.  Tensors may have any strides."""
    return RMSNormFunction.apply(x, weight, residual, eps, dropout, seed, offset, fp8)
