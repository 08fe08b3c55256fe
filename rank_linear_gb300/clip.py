"""Global gradient norm and clipping over many tensors: what stands between
the dA, dB of every LoRA layer and the optimiser (include/lora_clip.h)."""
from __future__ import annotations

import math

import torch

from . import _lib
from .lora import _dtype_code
from .rotary import _stream_on


class GradClip:
    """The plan over a list of gradient tensors, laid out once on the device.

    grads    contiguous CUDA tensors, bf16 and fp32 in any mix; None: those of
             `params`.  The plan holds their addresses: it keeps this memory and
             reads the values that are in it at each call.  Gradients have to
             stay there: zero_grad(set_to_none=False) or grad.zero_() between
             steps.  What zero_grad() does by default, dropping them for the
             next backward() to make new ones, leaves the plan with the old.
    out      tensors of the same shapes and types for the clipped gradients;
             None: in place.
    params   the parameters whose .grad these are, where that is to be made
             sure of: a call then raises if one of them has another gradient by
             now, or none, instead of clipping what is no longer in use.

    Calls that overlap on the GPU (other streams) need a plan each.
    """

    def __init__(self, grads=None, out=None, *, params=None):
        self.params = None if params is None else list(params)
        if grads is None:
            if params is None:
                raise ValueError("grads or params are needed")
            grads = [p.grad for p in self.params]
        self.grads = list(grads)
        if any(g is None for g in self.grads):
            raise ValueError("a parameter has no gradient yet")
        if self.params is not None and len(self.params) != len(self.grads):
            raise ValueError(f"{len(self.params)} parameters for {len(self.grads)} gradients")
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.out)} outputs for {len(self.grads)} gradients")
        table = (_lib.ClipTensor * max(len(self.grads), 1))()
        device = None
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            where = g.device
            if not g.is_cuda or not g.is_contiguous() or not o.is_contiguous():
                raise ValueError(f"gradient {i}: contiguous CUDA tensors are needed")
            if o is not g and (o.shape != g.shape or o.dtype != g.dtype or o.device != where):
                raise ValueError(f"gradient {i}: its output has another shape, type or device")
            if device is None:
                device = where
            elif where != device:
                raise ValueError(f"gradient {i} is on another device")
            row, at = table[i], g.data_ptr()
            row.in_ = at
            row.out = at if o is g else o.data_ptr()
            row.count, row.dtype = g.numel(), _dtype_code(g)
        L = _lib.lib()
        self.bytes = int(L.lora_clip_plan_bytes(table, len(self.grads)))
        if self.bytes == 0:
            _lib.check(_lib.LORA_ERR_INVALID_ARG, "lora_clip_plan_bytes")
        image = torch.empty(self.bytes, dtype=torch.uint8)
        _lib.check(L.lora_clip_plan_build(table, len(self.grads), image.data_ptr(), self.bytes),
                   "lora_clip_plan_build")
        self.plan = image.to(device if device is not None else torch.device("cuda"))
        self.device, self._at = self.plan.device, self.plan.data_ptr()
        # (a tensor may be given other memory: what the plan points to stays)
        self._memory = [t.detach() for t in (*self.grads, *self.out)]
        self._places = [g.data_ptr() for g in self.grads]
        self._check_params()
        self._scalar = torch.empty((), dtype=torch.float32, device=self.device)

    def _check_params(self):
        if self.params is not None:
            for i, (p, at) in enumerate(zip(self.params, self._places)):
                if p.grad is None or p.grad.data_ptr() != at:
                    raise RuntimeError(f"parameter {i} no longer has the gradient that the plan was made for: "
                                       "clear gradients in place (zero_grad(set_to_none=False))")

    @staticmethod
    def _largest(norm_type) -> int:
        if norm_type == 2 or norm_type == math.inf:
            return int(norm_type == math.inf)
        raise ValueError(f"norm_type = {norm_type} is not 2 or inf")

    def _norm_out(self, norm, stream):
        if norm is None:
            if stream is not None:
                with torch.cuda.stream(stream):
                    return torch.empty_like(self._scalar)
            return torch.empty_like(self._scalar)
        if norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != self.device:
            raise ValueError("norm must be one float32 on the gradients' device")
        return norm

    def norm(self, *, norm_type: float = 2.0, norm=None, stream=None):
        """The global norm (a device scalar); nothing is scaled."""
        self._check_params()
        norm = self._norm_out(norm, stream)
        st = _lib.lib().lora_clip_norm(self._at, self.bytes, self._largest(norm_type),
                                       norm.data_ptr(), _stream_on(self.device, stream))
        if st:
            _lib.check(st, "lora_clip_norm")
        return norm

    def clip(self, max_norm: float, *, norm_type: float = 2.0, norm=None, stream=None):
        """Scales every gradient by min(1, max_norm / (norm + 1e-6)); returns the
        norm before it (a device scalar)."""
        self._check_params()
        norm = self._norm_out(norm, stream)
        st = _lib.lib().lora_clip(self._at, self.bytes, float(max_norm), self._largest(norm_type),
                                  norm.data_ptr(), _stream_on(self.device, stream))
        if st:
            _lib.check(st, "lora_clip")
        return norm
