"""Attention between the q, k, v and o LoRA layers: scores capped by a tanh, a
bias that falls with distance, document and prefix masks; forward, backward,
and one new token over a cache (formulas in include/lora_attention.h; ch05
"Acceleration principles: Triton kernels and fused LoRA", §5.10).
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .lora import _ptr
from .rotary import _block, _empty_like, _layout, _on, _same_device, _stream_on


def _strides(t, name, device):
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
    _same_device(t, name, device)
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return s[:3]


def _check_word(t, dtype, name, shape, device):
    if t.dtype != dtype or not t.is_cuda or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor of shape {tuple(shape)}")
    _same_device(t, name, device)
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _make_shape(q, k, v, scale, causal, softcap, slopes, qd, kd, prefix, like_q, like_k):
    """The argument block without addresses; like_q, like_k: the other tensors
    by their names in it, of q's (k's) shape."""
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("q is [batch, q_len, q_heads, dim], k and v [batch, k_len, k_heads, dim]")
    b, sq, hq, d = q.shape
    sk, hk = k.shape[1], k.shape[2]
    if k.shape[0] != b or k.shape[3] != d:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not fit")
    sh = _lib.AttentionShape(batch=b, q_len=sq, k_len=sk, q_heads=hq, k_heads=hk, dim=d,
                             causal=int(causal), scale=d ** -0.5 if scale is None else scale,
                             softcap=softcap)
    on = q.device
    sh.q, sh.k, sh.v = _strides(q, "q", on), _strides(k, "k", on), _strides(v, "v", on)
    for like, others in ((q, like_q), (k, like_k)):
        for name, t in others.items():
            if t.shape != like.shape:
                raise ValueError(f"{name} {tuple(t.shape)} is not {tuple(like.shape)}")
            setattr(sh, name, _strides(t, name, on))
    if slopes is not None:
        _check_word(slopes, torch.float32, "slopes", (hq,), on)
    if qd is not None:
        _check_word(qd, torch.int32, "q documents", (b, sq), on)
        _check_word(kd, torch.int32, "k documents", (b, sk), on)
        sh.q_docs_stride, sh.k_docs_stride = qd.stride(0), kd.stride(0)
    if prefix is not None:
        _check_word(prefix, torch.int32, "prefix", (b,), on)
    return sh


def _options(scale, causal, softcap):
    """As plain numbers: a tensor's value is read at each call, as it is then (what
    is kept by layout is kept by these values too)."""
    return (None if scale is None else float(scale)), bool(causal), float(softcap or 0.0)


def _doc_pair(documents, q, k):
    """(queries' documents, keys')."""
    if documents is None:
        return None, None
    if isinstance(documents, (tuple, list)):
        if len(documents) != 2 or (documents[0] is None) != (documents[1] is None):
            raise ValueError("documents is one tensor, or the queries' and the keys'")
        return documents
    sq, sk = q.shape[1], k.shape[1]
    if sq > sk:
        raise ValueError("one documents tensor needs q_len <= k_len")
    return (documents if sq == sk else documents[:, sk - sq:]), documents


def _filled(block, slopes, qd, kd, prefix):
    """The block with this call's addresses."""
    if slopes is None and qd is None and prefix is None:
        return block
    sh = _lib.AttentionShape.from_buffer_copy(block)
    sh.slopes, sh.prefix = _ptr(slopes), _ptr(prefix)
    if qd is not None and qd.numel() and kd.numel():  # an empty side: nothing to mask
        sh.q_docs, sh.k_docs = _ptr(qd), _ptr(kd)
    return sh


def _workspace_bytes(sh, documents, prefix, backward):
    if documents or prefix:  # given or not: any address stands for them
        sh = _lib.AttentionShape.from_buffer_copy(sh)
        if documents:
            sh.q_docs = sh.k_docs = 16
        if prefix:
            sh.prefix = 16
    return _lib.lib().lora_attention_workspace_bytes(ctypes.byref(sh), backward)


def _scratch(nbytes, like, workspace):
    if workspace is not None:
        if workspace.device != like.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of q")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None


def _size(t):
    return 0 if t is None else t.numel() * t.element_size()


def attention_forward(q, k, v, *, scale=None, causal=False, softcap=0.0, slopes=None,
                      documents=None, prefix=None, out=None, lse=None, workspace=None,
                      stream=None):
    """(o, lse) of q [batch, q_len, q_heads, dim] over k, v [batch, k_len, k_heads, dim].

    scale      of the scores; None: dim ** -0.5.
    causal     the queries are the last q_len of the k_len positions.
    softcap    > 0: scores become softcap * tanh(score / softcap).
    slopes     float32 [q_heads]: score - slope * |distance|.
    documents  int32 [batch, k_len], the queries' being its last q_len (or a
               pair [batch, q_len], [batch, k_len]): a pair of tokens is
               visible within one document; below zero: padding.
    prefix     int32 [batch]: keys before it are visible to every query
               (with causal).
    """
    qd, kd = _doc_pair(documents, q, k)
    scale, causal, softcap = _options(scale, causal, softcap)
    with _on(stream):
        # (an output made here has the layout that q's decides)
        key = ("forward", _layout(q), _layout(k), _layout(v), _layout(out), scale, causal, softcap,
               _layout(slopes), _layout(qd), _layout(kd), _layout(prefix))
        if out is None:
            out = _empty_like(q)

        def make():
            sh = _make_shape(q, k, v, scale, causal, softcap, slopes, qd, kd, prefix,
                             {"o": out}, {})
            need = _workspace_bytes(sh, qd is not None, prefix is not None, 0)
            return sh, need, (sh.batch, sh.q_heads, sh.q_len)
        block, need, rows = _block(key, make)
        if lse is None:
            lse = torch.empty(rows, dtype=torch.float32, device=q.device)
        elif lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != rows or \
                lse.device != q.device:
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {rows}")
        workspace = _scratch(need, q, workspace)
    sh = _filled(block, slopes, qd, kd, prefix)
    st = _lib.lib().lora_attention_fwd(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                       _ptr(lse), _ptr(workspace), _size(workspace),
                                       _stream_on(q.device, stream))
    if st:
        _lib.check(st, "lora_attention_fwd")
    return out, lse


def attention_backward(dout, q, k, v, out, lse, *, scale=None, causal=False, softcap=0.0,
                       slopes=None, documents=None, prefix=None, dq=None, dk=None, dv=None,
                       workspace=None, stream=None):
    """(dq, dk, dv) from the gradient of attention_forward's output."""
    if lse.dtype != torch.float32 or not lse.is_contiguous() or \
            lse.shape != (q.shape[0], q.shape[2], q.shape[1]) or lse.device != q.device:
        raise ValueError("lse must be the forward's: float32 [batch, q_heads, q_len]")
    qd, kd = _doc_pair(documents, q, k)
    scale, causal, softcap = _options(scale, causal, softcap)
    with _on(stream):
        # (outputs made here have the layouts that q's, k's and v's decide, and
        # memory of their own: what keeps one of them does not keep the others)
        key = ("backward", _layout(q), _layout(k), _layout(v), _layout(out), _layout(dout),
               _layout(dq), _layout(dk), _layout(dv), scale, causal, softcap, _layout(slopes),
               _layout(qd), _layout(kd), _layout(prefix))
        dq = _empty_like(q) if dq is None else dq
        dk = _empty_like(k) if dk is None else dk
        dv = _empty_like(v) if dv is None else dv

        def make():
            sh = _make_shape(q, k, v, scale, causal, softcap, slopes, qd, kd, prefix,
                             {"o": out, "d_o": dout, "dq": dq}, {"dk": dk, "dv": dv})
            return sh, _workspace_bytes(sh, qd is not None, prefix is not None, 1)
        block, need = _block(key, make)
        workspace = _scratch(need, q, workspace)
    sh = _filled(block, slopes, qd, kd, prefix)
    st = _lib.lib().lora_attention_bwd(ctypes.byref(sh), _ptr(dout), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(out), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                                       _ptr(workspace), _size(workspace),
                                       _stream_on(q.device, stream))
    if st:
        _lib.check(st, "lora_attention_bwd")
    return dq, dk, dv


def attention_decode(q, k_cache, v_cache, lengths, *, scale=None, softcap=0.0, slopes=None,
                     out=None, workspace=None, stream=None):
    """One new token per sequence: q [batch, q_heads, dim] over the first
    lengths[b] (int32 [batch], the token itself included) of k_cache, v_cache
    [batch, positions, k_heads, dim].  Returns o like q; zero where the length is."""
    if q.dim() != 3:
        raise ValueError("q must be [batch, q_heads, dim]")
    L = _lib.lib()
    scale, _, softcap = _options(scale, False, softcap)
    with _on(stream):
        key = ("token", _layout(q), _layout(k_cache), _layout(v_cache), _layout(lengths), scale,
               softcap, _layout(slopes), _layout(out))
        if out is None:
            out = _empty_like(q)
        sh, need = _block(key, lambda: _make_token(q, k_cache, v_cache, lengths, scale, softcap,
                                                   slopes, out))
        sh = _filled(sh, slopes, None, None, None)
        workspace = _scratch(need, q, workspace)
    st = L.lora_attention_token(ctypes.byref(sh), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                _ptr(lengths), _ptr(out), _ptr(workspace), _size(workspace),
                                _stream_on(q.device, stream))
    if st:
        _lib.check(st, "lora_attention_token")
    return out


def _make_token(q, k_cache, v_cache, lengths, scale, softcap, slopes, out):
    if out.shape != q.shape:
        raise ValueError(f"out {tuple(out.shape)} is not {tuple(q.shape)}")
    _check_word(lengths, torch.int32, "lengths", (q.shape[0],), q.device)
    sh = _make_shape(q.unsqueeze(1), k_cache, v_cache, scale, False, softcap, slopes, None, None,
                     None, {"o": out.unsqueeze(1)}, {})
    return sh, _lib.lib().lora_attention_token_workspace_bytes(ctypes.byref(sh))


def _fit(t):
    """t itself where its strides suit the kernels, else a contiguous copy (of an
    expanded tensor too)."""
    ok = (t.stride(-1) == 1 or t.shape[-1] == 1) and t.data_ptr() % 16 == 0 and \
        all(n == 1 or (s > 0 and s % 8 == 0) for n, s in zip(t.shape[:3], t.stride()))
    # (contiguous() would give back a contiguous tensor at an odd address)
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class AttentionFunction(torch.autograd.Function):
    """Autograd function: saves q, k, v, the output and its log-sum-exp.  Gradients
    for q, k and v, once (not gradients of gradients); slopes are constants."""

    @staticmethod
    def forward(ctx, q, k, v, slopes, documents, prefix, scale, causal, softcap):
        q, k, v = _fit(q), _fit(k), _fit(v)
        # (the backward's are the forward's, whatever a tensor of them holds then)
        ctx.opts = dict(zip(("scale", "causal", "softcap"), _options(scale, causal, softcap)))
        pair = isinstance(documents, (tuple, list))
        docs = tuple(documents) if pair else (documents,)
        out, lse = attention_forward(q, k, v, slopes=slopes, documents=documents, prefix=prefix,
                                     **ctx.opts)
        ctx.save_for_backward(q, k, v, out, lse, slopes, prefix, *docs)
        ctx.pair = pair
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        if ctx.needs_input_grad[3]:
            raise RuntimeError("slopes get no gradient: give them detached")
        q, k, v, out, lse, slopes, prefix, *docs = ctx.saved_tensors
        dq, dk, dv = attention_backward(_fit(dout), q, k, v, out, lse, slopes=slopes,
                                        documents=tuple(docs) if ctx.pair else docs[0],
                                        prefix=prefix, **ctx.opts)
        return dq, dk, dv, None, None, None, None, None, None


def attention(q, k, v, *, scale=None, causal=False, softcap=0.0, slopes=None, documents=None,
              prefix=None):
    """attention_forward's output with gradients for q, k and v (whose strides may be
    any: what the kernels do not take as it is is copied).  Slopes are constants:
    a backward with slopes that require a gradient raises."""
    return AttentionFunction.apply(q, k, v, slopes, documents, prefix, scale, causal, softcap)
