"""Softmax cross entropy of a frozen head over a large vocabulary, with the
gradient of the hidden states and without keeping the logits (formulas in
include/lora_loss.h; ch05 "Acceleration principles: Triton kernels and fused
LoRA", §5.7)."""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .dropout import _collapsed
from .lora import _ptr
from .rotary import _block, _empty_like, _layout, _on, _same_device, _stream_on


def _check_matrix(t, name, device):
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
    _same_device(t, name, device)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")


def _make(X, W, targets, weights, softcap, mean, dX, losses):
    if X.dim() < 1 or W.dim() != 2 or X.shape[-1] != W.shape[1]:
        raise ValueError(f"X {tuple(X.shape)} and W {tuple(W.shape)} do not fit")
    lead = X.shape[:-1]
    _check_matrix(X, "X", X.device)
    _check_matrix(W, "W", X.device)
    if targets.dtype not in (torch.int32, torch.int64) or targets.shape != lead or \
            not targets.is_contiguous():
        raise ValueError(f"targets must be a contiguous int32 or int64 tensor of shape {tuple(lead)}")
    _same_device(targets, "targets", X.device)
    for name, t in (("weights", weights), ("losses", losses)):
        if t is None:
            continue
        if t.dtype != torch.float32 or t.shape != lead or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(lead)}")
        _same_device(t, name, X.device)
    steps = [_collapsed(lead, X.stride()[:-1]), 0]
    if dX is not None:
        _check_matrix(dX, "dX", X.device)
        if dX.shape != X.shape:
            raise ValueError(f"dX {tuple(dX.shape)} is not {tuple(X.shape)}")
        steps[1] = _collapsed(lead, dX.stride()[:-1])
    if None in steps:
        raise ValueError("the rows of X and dX must lie one stride apart")
    sh = _lib.LossShape(rows=lead.numel(), vocab=W.shape[0], dim=W.shape[1],
                        target_bits=64 if targets.dtype == torch.int64 else 32, mean=int(mean),
                        softcap=softcap, x=steps[0], w=W.stride(0), dx=steps[1])
    need = _lib.lib().lora_loss_workspace_bytes(ctypes.byref(sh), int(dX is not None))
    return sh, need


def _workspace(workspace, need, X):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=X.device) if need else None
    if workspace.device != X.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of X")
    return workspace


def cross_entropy_forward(X, W, targets, *, weights=None, softcap=0.0, reduction="mean",
                          gradient=False, loss=None, losses=None, dX=None, workspace=None,
                          stream=None):
    """(loss, losses, dX or None) of hidden states X [..., dim] under a head W
    [vocab, dim], both bf16: the logits are X W^T, capped by softcap * tanh(z / softcap)
    where softcap > 0.

    targets    int32 or int64 [...]; below 0: the token does not count (and costs
               nothing).  At or beyond the vocabulary: NaN.
    weights    float32 [...]: of each token in the loss; None: 1.
    reduction  "mean": by the sum of the weights of the tokens that count, "sum".
    gradient   also returns dX, the gradient of loss (W is frozen).
    loss, losses  float32: the reduced one, and each token's own (0 where it does
               not count); -losses are the targets' log-probabilities.
    dX         may be X (in place).
    """
    if reduction not in ("mean", "sum"):
        raise ValueError(f"reduction {reduction!r} is not 'mean' or 'sum'")
    gradient, softcap = bool(gradient) or dX is not None, float(softcap or 0.0)
    if softcap != 0.0 and not 2.0 ** -100 <= softcap <= 2.0 ** 100:
        raise ValueError(f"softcap = {softcap} is not 0 or within 2^-100 .. 2^100")
    # (outputs made here have the layouts that X's decides)
    key = ("loss", _layout(X), _layout(W), _layout(targets), _layout(weights), _layout(dX),
           _layout(losses), softcap, reduction, gradient)
    if loss is not None and (loss.dtype != torch.float32 or loss.numel() != 1 or loss.device != X.device):
        raise ValueError("loss must be one float32 on the device of X")

    def buffers():
        return (torch.empty((), dtype=torch.float32, device=X.device) if loss is None else loss,
                torch.empty(X.shape[:-1], dtype=torch.float32, device=X.device) if losses is None else losses,
                _empty_like(X) if gradient and dX is None else dX)

    def make():
        return _make(X, W, targets, weights, softcap, reduction == "mean", dX, losses)
    if stream is None:
        loss, losses, dX = buffers()
        sh, need = _block(key, make)
        workspace = _workspace(workspace, need, X)
    else:
        with _on(stream):
            loss, losses, dX = buffers()
            sh, need = _block(key, make)
            workspace = _workspace(workspace, need, X)
    st = _lib.lib().lora_loss(ctypes.byref(sh), _ptr(X), _ptr(W), _ptr(targets), _ptr(weights),
                              _ptr(loss), _ptr(losses), _ptr(dX), _ptr(workspace),
                              0 if workspace is None else workspace.numel() * workspace.element_size(),
                              _stream_on(X.device, stream))
    if st:
        _lib.check(st, "lora_loss")
    return loss, losses, dX


def cross_entropy_backward(dloss, dX, *, out=None, stream=None):
    """dloss (one float32 on the device) times the dX of cross_entropy_forward, rounded
    once more; out may be dX."""
    if dloss.dtype != torch.float32 or dloss.numel() != 1 or not dloss.is_cuda:
        raise ValueError("dloss must be one float32 on the device")
    _same_device(dloss, "dloss", dX.device)
    with _on(stream):
        if out is None:
            out = _empty_like(dX)

    def make():
        steps = []
        for name, t in (("dX", dX), ("out", out)):
            _check_matrix(t, name, dX.device)
            steps.append(_collapsed(t.shape[:-1], t.stride()[:-1]))
        if out.shape != dX.shape or None in steps:
            raise ValueError("out must be like dX, the rows of both one stride apart")
        return _lib.LossShape(rows=dX.shape[:-1].numel(), vocab=1, dim=dX.shape[-1], target_bits=64,
                              x=steps[1], w=dX.shape[-1], dx=steps[0])
    sh = _block(("loss scale", _layout(dX), _layout(out)), make)
    st = _lib.lib().lora_loss_scale(ctypes.byref(sh), _ptr(dX), _ptr(dloss), _ptr(out),
                                    _stream_on(dX.device, stream))
    if st:
        _lib.check(st, "lora_loss_scale")
    return out


def _fit(t):
    """t itself where its rows suit the kernels, else a contiguous copy."""
    step = _collapsed(t.shape[:-1], t.stride()[:-1])
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and step is not None and \
        (t.shape[:-1].numel() <= 1 or (step % 8 == 0 and step >= t.shape[-1]))
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class CrossEntropyFunction(torch.autograd.Function):
    """Autograd function: makes the gradient of X beside the loss, where X wants one,
    and keeps that alone.  Gradients once (not gradients of gradients)."""

    @staticmethod
    def forward(ctx, X, W, targets, weights, softcap, reduction):
        loss, losses, dX = cross_entropy_forward(
            _fit(X), _fit(W), targets.contiguous(),
            weights=None if weights is None else weights.contiguous(),
            softcap=softcap, reduction=reduction, gradient=ctx.needs_input_grad[0])
        ctx.save_for_backward(dX)
        ctx.mark_non_differentiable(losses)
        return loss, losses

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        if ctx.needs_input_grad[1] or ctx.needs_input_grad[3]:
            raise RuntimeError("the head and the weights get no gradient: give them detached")
        dX, = ctx.saved_tensors
        return cross_entropy_backward(dloss, dX), None, None, None, None, None


def cross_entropy(X, W, targets, *, weights=None, softcap=0.0, reduction="mean"):
    """(loss, losses) of cross_entropy_forward, loss with the gradient of X (of any
    strides); losses are values without a gradient.  W and the weights are
    constants: a backward with one that requires a gradient raises."""
    if not torch.is_grad_enabled():
        X = X.detach()  # (its gradient is made with the loss: not where none is taken)
    return CrossEntropyFunction.apply(X, W, targets, weights, softcap, reduction)
