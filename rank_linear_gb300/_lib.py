"""ctypes binding of the C ABI in include/lora_linear.h (marshalling only).

The library is required: loading fails loudly if `liblora_linear.so` has not
been built; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblora_linear.so")

LORA_OK, LORA_ERR_INVALID_ARG, LORA_ERR_UNSUPPORTED, LORA_ERR_WORKSPACE, \
    LORA_ERR_CUDA, LORA_ERR_TIMEOUT = range(6)
LORA_BF16, LORA_FP32 = 0, 1
KERNEL_KINDS = ["prep", "down_fwd", "main_fwd", "down_bwd", "main_bwd", "grad_a", "grad_b",
                "down_bwd_grad_b", "swiglu_grad", "quant", "grad_a_b", "rotary", "grad_norm",
                "grad_clip", "attn_prep", "attn_fwd", "attn_dq", "attn_dkv", "attn_token", "norm",
                "norm_bwd", "dropout", "loss_prep", "loss_logits", "loss_rows", "loss_grad"]

_vp, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_int, _f32 = ctypes.c_int, ctypes.c_float

_i32 = ctypes.c_int32


class RotaryShape(ctypes.Structure):
    """lora_rotary_t"""
    _fields_ = [("batch", _i64), ("seq", _i64), ("q_heads", _i32), ("k_heads", _i32),
                ("dim", _i32), ("rot", _i32), ("interleaved", _i32), ("inverse", _i32),
                ("position_bits", _i32), ("magnitude", _f32), ("q_in", _i64 * 3),
                ("k_in", _i64 * 3), ("q_out", _i64 * 3), ("k_out", _i64 * 3),
                ("position", _i64 * 2)]


class ClipTensor(ctypes.Structure):
    """lora_clip_tensor_t"""
    _fields_ = [("in_", _vp), ("out", _vp), ("count", _i64), ("dtype", _i32)]


class AttentionShape(ctypes.Structure):
    """lora_attention_t"""
    _fields_ = [("batch", _i64), ("q_len", _i64), ("k_len", _i64), ("q_heads", _i32),
                ("k_heads", _i32), ("dim", _i32), ("causal", _i32), ("scale", _f32),
                ("softcap", _f32), ("q", _i64 * 3), ("k", _i64 * 3), ("v", _i64 * 3),
                ("o", _i64 * 3), ("d_o", _i64 * 3), ("dq", _i64 * 3), ("dk", _i64 * 3),
                ("dv", _i64 * 3), ("slopes", _vp), ("q_docs", _vp), ("k_docs", _vp),
                ("q_docs_stride", _i64), ("k_docs_stride", _i64), ("prefix", _vp)]


class Dropout(ctypes.Structure):
    """lora_dropout_t"""
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint32),
                ("state", _vp)]


class NormShape(ctypes.Structure):
    """lora_norm_t"""
    _fields_ = [("outer", _i64), ("inner", _i64), ("dim", _i32), ("weight_fp32", _i32),
                ("eps", _f32), ("x", _i64 * 2), ("residual", _i64 * 2), ("h", _i64 * 2),
                ("y", _i64 * 2), ("dy", _i64 * 2), ("dh", _i64 * 2), ("dx", _i64 * 2),
                ("dresidual", _i64 * 2)]


class LossShape(ctypes.Structure):
    """lora_loss_t"""
    _fields_ = [("rows", _i64), ("vocab", _i64), ("dim", _i32), ("target_bits", _i32),
                ("mean", _i32), ("softcap", _f32), ("x", _i64), ("w", _i64), ("dx", _i64)]


SIGNATURES = {
    "lora_linear_saved_bytes": ([_i64, _int, _int], _sz),
    "lora_linear_workspace_bytes": ([_i64, _i64, _i64, _int, _int], _sz),
    "lora_linear_fwd": ([_vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _int,
                         _vp, _vp, _vp, _sz, _vp], _int),
    "lora_linear_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _int,
                         _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "lora_linear_bwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64,
                                 _int, _vp, _vp, _vp, _vp], _int),
    "lora_status_string": ([_int], ctypes.c_char_p),
    "lora_last_error": ([], ctypes.c_char_p),
    "lora_device_status": ([_int], _int),
    "lora_launch_count": ([], ctypes.c_uint64),
    "lora_set_timing_events": ([ctypes.POINTER(_vp), ctypes.POINTER(_int), _int], _int),
    "lora_debug_withhold_arrive": ([_int], _int),
    "lora_debug_gemm_width": ([_int], _int),
    "lora_debug_withhold_gemm_stage": ([_int], _int),
    "lora_timing_used": ([], _int),
    "lora_fp8_quantize_w_workspace_bytes": ([], _sz),
    "lora_fp8_quantize_w": ([_vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "lora_fp8_quantize_rows": ([_vp, _i64, _i64, _vp, _vp, _vp], _int),
    "lora_fp8_workspace_bytes": ([_i64, _i64, _i64, _int], _sz),
    "lora_fp8_fwd": ([_vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                      _sz, _vp], _int),
    "lora_fp8_fwd_rows": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _vp,
                           _vp, _vp, _sz, _vp], _int),
    "lora_fp8_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _vp,
                      _vp, _vp, _vp, _sz, _vp], _int),
    "lora_q4_quantize_w": ([_vp, _i64, _i64, _vp, _vp, _vp], _int),
    "lora_q4_dequantize_w": ([_vp, _vp, _i64, _i64, _vp, _vp], _int),
    "lora_q4_fwd": ([_vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _vp, _vp, _vp, _sz,
                     _vp], _int),
    "lora_q4_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _vp, _vp,
                     _vp, _vp, _sz, _vp], _int),
    "lora_swiglu_saved_bytes": ([_i64, _i64, _int], _sz),
    "lora_swiglu_workspace_bytes": ([_i64, _i64, _i64, _int], _sz),
    "lora_swiglu_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64, _i64, _int,
                         _vp, _vp, _vp, _sz, _vp], _int),
    "lora_swiglu_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _int, _i64, _i64,
                         _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "lora_rotary_turns": ([_vp, _int, _vp], _int),
    "lora_rotary": ([_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp], _int),
    "lora_clip_plan_bytes": ([_vp, _int], _sz),
    "lora_clip_plan_build": ([_vp, _int, _vp, _sz], _int),
    "lora_clip_norm": ([_vp, _sz, _int, _vp, _vp], _int),
    "lora_clip": ([_vp, _sz, _f32, _int, _vp, _vp], _int),
    "lora_attention_workspace_bytes": ([_vp, _int], _sz),
    "lora_attention_fwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "lora_attention_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
                           _int),
    "lora_attention_token_workspace_bytes": ([_vp], _sz),
    "lora_dropout": ([_vp, _i64, _i64, _i64, _i64, _vp, _int, _vp, _vp], _int),
    "lora_norm_fwd": ([_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp], _int),
    "lora_norm_workspace_bytes": ([_vp, _int], _sz),
    "lora_norm_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _sz, _vp],
                      _int),
    "lora_loss_workspace_bytes": ([_vp, _int], _sz),
    "lora_loss": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "lora_loss_scale": ([_vp, _vp, _vp, _vp, _vp], _int),
    "lora_attention_token": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
}

_lib = None
_lock = threading.Lock()


class LoraError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def lib():
    """The loaded library (built on first use if sources are present)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m rank_linear_gb300.build` "
                    "(nvcc, sm_103a); there is no CPU or PyTorch fallback")
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = res
            _lib = L
        return _lib


def check(status: int, what: str = "lora call") -> None:
    if status != LORA_OK:
        L = lib()
        name = L.lora_status_string(status).decode()
        detail = L.lora_last_error().decode()
        raise LoraError(status, f"{what}: {name}: {detail}")
