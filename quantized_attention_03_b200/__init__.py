"""Python binding of libsage.so, the B200 (sm_100a) SageAttention forward pass.

The C entry points declared in ``include/sage.h`` are exposed under the same names and
argument order (``sage_attn_fwd(q, k, v, out, B, H, N, d, causal, smooth_k, pv_mode,
sm_scale, stream)`` ...). Pointer arguments accept torch tensors (their device
pointer), plain integers or ``None``; ``stream=None`` means torch's current stream.
This module only marshals arguments: every step of the computation runs in the CUDA
library, and nothing falls back to another implementation. If the library is missing
the first call raises.

Convenience wrappers (``sageattn``, ``sageattn_varlen``, ``quant_qk``, ...) allocate
the output tensors with torch and call the same entry points.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsage.so")

SAGE_OK = 0
SAGE_ERR_INVALID_ARG = 1
SAGE_ERR_UNSUPPORTED = 2
SAGE_ERR_MISALIGNED = 3
SAGE_ERR_WORKSPACE = 4
SAGE_ERR_CUDA = 5
SAGE_ERR_TIMEOUT = 6
SAGE_ERR_BAD_SEQLENS = 7
SAGE_ERR_BAD_PAGE = 8
SAGE_PV_FP16 = 0
SAGE_PV_FP8 = 1
SAGE_SMOOTH_K = 1     # flags of the fused entry points' smooth_k argument
SAGE_SMOOTH_V = 2
SAGE_SMOOTH_Q = 4
SAGE_QK_FINE = 8
SAGE_F16 = 0          # dtype of the rotary and 4-bit cache entry points
SAGE_BF16 = 1
SAGE_ROPE_INTERLEAVED = 1   # flags of the rotations
SAGE_ROPE_INVERSE = 2
SAGE_ROPE_PLAIN = 0         # scalings of sage_rope_freqs
SAGE_ROPE_LINEAR = 1
SAGE_ROPE_BASE = 2
SAGE_ROPE_PARTS = 3

Q_BLOCK = 128
K_BLOCK = 64
DECODE_MAX_Q = 16   # SAGE_DECODE_MAX_Q: most queries sage_attn_decode_quantized takes

# name -> (restype, argtypes) as declared in include/sage.h
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_D = ctypes.c_double
_L = ctypes.c_int64
_Z = ctypes.c_size_t
_S = ctypes.c_int  # sage_status_t
SIGNATURES = {
    "sage_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "sage_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sage_workspace_size_kv": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "sage_quant_qk_kv": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _Z,
                              _P]),
    "sage_attn_fwd_kv": (_S, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _Z, _P]),
    "sage_attn_varlen_fwd_kv": (_S, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                     _I, _F, _P, _Z, _P]),
    "sage_attn_fwd_quantized_kv": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                        _I, _I, _F, _I, _P]),
    "sage_attn_decode_workspace_size": (_Z, [_I, _I, _I, _I, _I]),
    "sage_attn_decode_quantized": (_S, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                                        _P, _Z, _P]),
    "sage_rope_freqs": (_S, [_P, _P, _I, _D, _I, _D, _D, _D, _D]),
    "sage_rope": (_S, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _L, _P, _D, _I, _P]),
    "sage_kv4_page_bytes": (_Z, [_I, _I]),
    "sage_kv4_append": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                             _I, _I, _P, _D, _I, _P]),
    "sage_kv4_gather": (_S, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P]),
    "sage_attn_kv4_workspace_size": (_Z, [_I, _I, _I, _I]),
    "sage_attn_kv4": (_S, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                           _F, _P, _P, _Z, _P]),
    "sage_quant_qk": (_S, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "sage_quant_qk_ws": (_S, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "sage_quant_qk_varlen": (_S, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P]),
    "sage_quant_v_fp8": (_S, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "sage_quant_v_fp8_varlen": (_S, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "sage_quant_v_fp8_smooth": (_S, [_P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "sage_quant_v_fp8_ws": (_S, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P]),
    "sage_quant_v_fp8_smooth_varlen": (_S, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "sage_attn_fwd": (_S, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P]),
    "sage_attn_fwd_ws": (_S, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _Z, _P]),
    "sage_attn_varlen_fwd": (_S, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                  _Z, _P]),
    "sage_attn_fwd_quantized": (_S, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F,
                                     _P]),
    "sage_attn_fwd_quantized_smooth_v": (_S, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                              _I, _F, _P]),
    "sage_debug_qk_int32": (_S, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "sage_attn_fwd_noalloc": (_S, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P]),
    "sage_debug_wait_timeout": (_S, [ctypes.c_ulonglong, _P]),
    "sage_get_device_status": (_S, [_P]),
    "sage_status_string": (ctypes.c_char_p, [_I]),
    "sage_last_cuda_error": (_I, []),
    "sage_version": (_I, []),
}

_lib = None


class SageError(RuntimeError):
    def __init__(self, name: str, code: int):
        self.code = code
        msg = status_string(code) if _lib is not None else str(code)
        super().__init__(f"{name} failed: {msg} ({code})")


def lib() -> ctypes.CDLL:
    """Load libsage.so (built in-tree by ``build.py``); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m quantized_attention_03_b200.build`"
                " (there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().sage_status_string(int(code)).decode()


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _call(name: str, *args):
    rc = getattr(lib(), name)(*args)
    if rc != SAGE_OK:
        raise SageError(name, rc)
    return rc


# ---------------------------------------------------------------- C-ABI names


def sage_workspace_size(nseq, H, max_seqlen, total_tokens, d, pv_mode) -> int:
    return int(lib().sage_workspace_size(nseq, H, max_seqlen, total_tokens, d, pv_mode))


def sage_attn_workspace_size(B, H, N, d, pv_mode) -> int:
    return int(lib().sage_attn_workspace_size(B, H, N, d, pv_mode))


def sage_workspace_size_kv(nseq, H, max_seqlen_q, max_seqlen_k, total_q, total_k, d,
                           pv_mode) -> int:
    return int(lib().sage_workspace_size_kv(nseq, H, max_seqlen_q, max_seqlen_k, total_q, total_k,
                                            d, pv_mode))


def sage_quant_qk_kv(q, k, q_i8, q_scale, k_i8, k_scale, k_mean, q_mean, q_comp, B, H, Nq, Nk,
                     d, flags, workspace=None, ws_bytes=0, stream=None):
    return _call("sage_quant_qk_kv", _ptr(q), _ptr(k), _ptr(q_i8), _ptr(q_scale), _ptr(k_i8),
                 _ptr(k_scale), _ptr(k_mean), _ptr(q_mean), _ptr(q_comp), B, H, Nq, Nk, d,
                 int(flags), _ptr(workspace), int(ws_bytes), _stream(stream))


def sage_attn_fwd_kv(q, k, v, out, B, H, Nq, Nk, d, causal, smooth_k, pv_mode, sm_scale,
                     workspace=None, ws_bytes=0, stream=None):
    return _call("sage_attn_fwd_kv", _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, Nq, Nk, d,
                 int(causal), int(smooth_k), int(pv_mode), float(sm_scale), _ptr(workspace),
                 int(ws_bytes), _stream(stream))


def sage_attn_varlen_fwd_kv(q, k, v, out, cu_seqlens_q, cu_seqlens_k, nseq, total_q, total_k,
                            max_seqlen_q, max_seqlen_k, H, d, causal, smooth_k, pv_mode, sm_scale,
                            workspace=None, ws_bytes=0, stream=None):
    return _call("sage_attn_varlen_fwd_kv", _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                 _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), nseq, total_q, total_k, max_seqlen_q,
                 max_seqlen_k, H, d, int(causal), int(smooth_k), int(pv_mode), float(sm_scale),
                 _ptr(workspace), int(ws_bytes), _stream(stream))


def sage_attn_decode_workspace_size(B, H, Nq, Nk, d) -> int:
    return int(lib().sage_attn_decode_workspace_size(B, H, Nq, Nk, d))


def sage_attn_decode_quantized(q_i8, q_scale, k_i8, k_scale, v, out, B, H, Nq, Nk, d, causal,
                               sm_scale, flags, workspace, ws_bytes, stream=None):
    return _call("sage_attn_decode_quantized", _ptr(q_i8), _ptr(q_scale), _ptr(k_i8),
                 _ptr(k_scale), _ptr(v), _ptr(out), B, H, Nq, Nk, d, int(causal),
                 float(sm_scale), int(flags), _ptr(workspace), int(ws_bytes), _stream(stream))


def _i64s(x):
    """A host array of int64 (or None) as sage.h's strides arguments take it."""
    return None if x is None else (ctypes.c_int64 * len(x))(*x)


def sage_rope_freqs(freqs, mscale, rot_dim, base, scaling, factor, original_len, beta_fast,
                    beta_slow):
    """freqs, mscale: host addresses (int, ctypes array or CPU tensor; mscale may be None)."""
    freqs = freqs if isinstance(freqs, ctypes.Array) else _ptr(freqs)
    return _call("sage_rope_freqs", freqs,
                 mscale if isinstance(mscale, ctypes.Array) else _ptr(mscale), rot_dim,
                 float(base), int(scaling), float(factor), float(original_len), float(beta_fast),
                 float(beta_slow))


def sage_rope(q, q_out, k, k_out, positions, freqs, dtype, B, N, Hq, Hk, d, rot_dim, pos_stride,
              strides, mscale, flags, stream=None):
    """strides: 12 integers or None (see sage.h)."""
    return _call("sage_rope", _ptr(q), _ptr(q_out), _ptr(k), _ptr(k_out), _ptr(positions),
                 _ptr(freqs), dtype, B, N, Hq, Hk, d, rot_dim, pos_stride, _i64s(strides), mscale,
                 flags, _stream(stream))


def sage_kv4_page_bytes(page_size, d) -> int:
    return int(lib().sage_kv4_page_bytes(page_size, d))


def sage_kv4_append(cache, block_table, kv_lens, cu_seqlens, k, v, q, q_out, freqs, k_mean, dtype,
                    nseq, total, Hq, Hkv, d, page_size, num_pages, max_pages, rot_dim, strides,
                    mscale, flags, stream=None):
    """strides: 8 integers or None (see sage.h)."""
    return _call("sage_kv4_append", _ptr(cache), _ptr(block_table), _ptr(kv_lens),
                 _ptr(cu_seqlens), _ptr(k), _ptr(v), _ptr(q), _ptr(q_out), _ptr(freqs),
                 _ptr(k_mean), dtype, nseq, total, Hq, Hkv, d, page_size, num_pages, max_pages,
                 rot_dim, _i64s(strides), mscale, flags, _stream(stream))


def sage_kv4_gather(cache, block_table, kv_lens, cu_seqlens, k_out, v_out, dtype, nseq, total, Hkv,
                    rep, d, page_size, num_pages, max_pages, stream=None):
    return _call("sage_kv4_gather", _ptr(cache), _ptr(block_table), _ptr(kv_lens),
                 _ptr(cu_seqlens), _ptr(k_out), _ptr(v_out), dtype, nseq, total, Hkv, rep, d,
                 page_size, num_pages, max_pages, _stream(stream))


def sage_attn_kv4_workspace_size(Hq, Hkv, max_q, d) -> int:
    return int(lib().sage_attn_kv4_workspace_size(Hq, Hkv, max_q, d))


def sage_attn_kv4(q, cache, block_table, kv_lens, cu_seqlens, out, lse, dtype, nseq, total, max_q,
                  Hq, Hkv, d, page_size, num_pages, max_pages, causal, sm_scale, q_strides,
                  workspace, ws_bytes, stream=None):
    """q_strides: 2 integers or None (see sage.h)."""
    return _call("sage_attn_kv4", _ptr(q), _ptr(cache), _ptr(block_table), _ptr(kv_lens),
                 _ptr(cu_seqlens), _ptr(out), _ptr(lse), dtype, nseq, total, max_q, Hq, Hkv, d,
                 page_size, num_pages, max_pages, int(causal), float(sm_scale), _i64s(q_strides),
                 _ptr(workspace), ws_bytes, _stream(stream))


def sage_attn_fwd_quantized_kv(q_i8, q_scale, k_i8, k_scale, v, v_scale, v_mean, q_comp, out, B,
                               H, Nq, Nk, d, causal, pv_mode, sm_scale, flags=0, stream=None):
    return _call("sage_attn_fwd_quantized_kv", _ptr(q_i8), _ptr(q_scale), _ptr(k_i8),
                 _ptr(k_scale), _ptr(v), _ptr(v_scale), _ptr(v_mean), _ptr(q_comp), _ptr(out), B,
                 H, Nq, Nk, d, int(causal), int(pv_mode), float(sm_scale), int(flags),
                 _stream(stream))


def sage_quant_qk(q, k, q_i8, q_scale, k_i8, k_scale, k_mean, B, H, N, d, smooth_k, stream=None):
    return _call("sage_quant_qk", _ptr(q), _ptr(k), _ptr(q_i8), _ptr(q_scale), _ptr(k_i8),
                 _ptr(k_scale), _ptr(k_mean), B, H, N, d, int(smooth_k), _stream(stream))


def sage_quant_qk_ws(q, k, q_i8, q_scale, k_i8, k_scale, k_mean, B, H, N, d, smooth_k, workspace,
                     ws_bytes, stream=None):
    return _call("sage_quant_qk_ws", _ptr(q), _ptr(k), _ptr(q_i8), _ptr(q_scale), _ptr(k_i8),
                 _ptr(k_scale), _ptr(k_mean), B, H, N, d, int(smooth_k), _ptr(workspace),
                 int(ws_bytes), _stream(stream))


def sage_quant_qk_varlen(q, k, cu_seqlens, nseq, total_tokens, max_seqlen, H, d, q_i8, q_scale,
                         k_i8, k_scale, k_mean, smooth_k, stream=None):
    return _call("sage_quant_qk_varlen", _ptr(q), _ptr(k), _ptr(cu_seqlens), nseq, total_tokens,
                 max_seqlen, H, d, _ptr(q_i8), _ptr(q_scale), _ptr(k_i8), _ptr(k_scale),
                 _ptr(k_mean), int(smooth_k), _stream(stream))


def sage_quant_v_fp8(v, v_e4m3, v_scale, B, H, N, d, stream=None):
    return _call("sage_quant_v_fp8", _ptr(v), _ptr(v_e4m3), _ptr(v_scale), B, H, N, d,
                 _stream(stream))


def sage_quant_v_fp8_varlen(v, cu_seqlens, nseq, total_tokens, max_seqlen, H, d, v_e4m3,
                            v_scale, stream=None):
    return _call("sage_quant_v_fp8_varlen", _ptr(v), _ptr(cu_seqlens), nseq, total_tokens,
                 max_seqlen, H, d, _ptr(v_e4m3), _ptr(v_scale), _stream(stream))


def sage_quant_v_fp8_ws(v, v_e4m3, v_scale, v_mean, B, H, N, d, workspace, ws_bytes,
                        stream=None):
    return _call("sage_quant_v_fp8_ws", _ptr(v), _ptr(v_e4m3), _ptr(v_scale), _ptr(v_mean), B, H,
                 N, d, _ptr(workspace), int(ws_bytes), _stream(stream))


def sage_quant_v_fp8_smooth(v, v_e4m3, v_scale, v_mean, B, H, N, d, stream=None):
    return _call("sage_quant_v_fp8_smooth", _ptr(v), _ptr(v_e4m3), _ptr(v_scale), _ptr(v_mean),
                 B, H, N, d, _stream(stream))


def sage_quant_v_fp8_smooth_varlen(v, cu_seqlens, nseq, total_tokens, max_seqlen, H, d, v_e4m3,
                                   v_scale, v_mean, stream=None):
    return _call("sage_quant_v_fp8_smooth_varlen", _ptr(v), _ptr(cu_seqlens), nseq,
                 total_tokens, max_seqlen, H, d, _ptr(v_e4m3), _ptr(v_scale), _ptr(v_mean),
                 _stream(stream))


def sage_attn_fwd(q, k, v, out, B, H, N, d, causal, smooth_k, pv_mode, sm_scale, stream=None):
    return _call("sage_attn_fwd", _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, N, d, int(causal),
                 int(smooth_k), int(pv_mode), float(sm_scale), _stream(stream))


def sage_attn_fwd_ws(q, k, v, out, B, H, N, d, causal, smooth_k, pv_mode, sm_scale, workspace,
                     ws_bytes, stream=None):
    return _call("sage_attn_fwd_ws", _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, N, d,
                 int(causal), int(smooth_k), int(pv_mode), float(sm_scale), _ptr(workspace),
                 int(ws_bytes), _stream(stream))


def sage_attn_varlen_fwd(q, k, v, out, cu_seqlens, nseq, total_tokens, max_seqlen, H, d, causal,
                         smooth_k, pv_mode, sm_scale, workspace=None, ws_bytes=0, stream=None):
    return _call("sage_attn_varlen_fwd", _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cu_seqlens),
                 nseq, total_tokens, max_seqlen, H, d, int(causal), int(smooth_k), int(pv_mode),
                 float(sm_scale), _ptr(workspace), int(ws_bytes), _stream(stream))


def sage_attn_fwd_quantized(q_i8, q_scale, k_i8, k_scale, v, v_scale, out, B, H, N, d, causal,
                            pv_mode, sm_scale, stream=None):
    return _call("sage_attn_fwd_quantized", _ptr(q_i8), _ptr(q_scale), _ptr(k_i8), _ptr(k_scale),
                 _ptr(v), _ptr(v_scale), _ptr(out), B, H, N, d, int(causal), int(pv_mode),
                 float(sm_scale), _stream(stream))


def sage_attn_fwd_quantized_smooth_v(q_i8, q_scale, k_i8, k_scale, v_e4m3, v_scale, v_mean, out,
                                     B, H, N, d, causal, sm_scale, stream=None):
    return _call("sage_attn_fwd_quantized_smooth_v", _ptr(q_i8), _ptr(q_scale), _ptr(k_i8),
                 _ptr(k_scale), _ptr(v_e4m3), _ptr(v_scale), _ptr(v_mean), _ptr(out), B, H, N,
                 d, int(causal), float(sm_scale), _stream(stream))


def sage_debug_qk_int32(q_i8, k_i8, s_out, B, H, N, d, stream=None):
    return _call("sage_debug_qk_int32", _ptr(q_i8), _ptr(k_i8), _ptr(s_out), B, H, N, d,
                 _stream(stream))


def sage_attn_fwd_noalloc(q, k, v, out, B, H, N, d, causal, smooth_k, pv_mode, sm_scale,
                          stream=None):
    """sage_attn_fwd with the library's static scratch (no allocation; see sage.h)."""
    return _call("sage_attn_fwd_noalloc", _ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, N, d,
                 int(causal), int(smooth_k), int(pv_mode), float(sm_scale), _stream(stream))


def sage_debug_wait_timeout(timeout_ns, stream=None):
    return _call("sage_debug_wait_timeout", int(timeout_ns), _stream(stream))


def sage_get_device_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status code."""
    return int(lib().sage_get_device_status(_stream(stream)))


def sage_status_string(code: int) -> str:
    return status_string(code)


def sage_last_cuda_error() -> int:
    return int(lib().sage_last_cuda_error())


def sage_version() -> int:
    return int(lib().sage_version())


# ------------------------------------------------------------ torch conveniences


def _check_status(stream=None):
    code = sage_get_device_status(stream)
    if code != SAGE_OK:
        raise SageError("device", code)


def _smooth_flags(smooth_k: bool, smooth_v: bool, fine: bool = False,
                  smooth_q: bool = False) -> int:
    return ((SAGE_SMOOTH_K if smooth_k else 0) | (SAGE_SMOOTH_V if smooth_v else 0)
            | (SAGE_QK_FINE if fine else 0) | (SAGE_SMOOTH_Q if smooth_q else 0))


def _want_fp16(*tensors):
    """What goes to the attention and quantization kernels by address alone is contiguous float16."""
    import torch
    for x in tensors:
        if x is not None and (x.dtype is not torch.float16 or not x.is_contiguous()):
            raise ValueError(f"contiguous float16 tensors are wanted, got {x.dtype} {tuple(x.shape)} with "
                             f"strides {x.stride()}")


def _want_size(name: str, x, n: int, like=None):
    """x holds the n elements that a kernel takes from its address on; more only as further rows
    of packed tensors like `like`."""
    if x.numel() != n and not (like is not None and x.numel() > n and x.shape[1:] == like.shape[1:]):
        raise ValueError(f"{name} of {n} elements is wanted (k and v with q's heads and channels), got "
                         f"{tuple(x.shape)}")


def _want_out(out, q):
    _want_fp16(out)
    if out.numel() < q.numel():
        raise ValueError(f"out has q's shape, got {tuple(out.shape)} and {tuple(q.shape)}")


def sageattn(q, k, v, causal: bool = False, smooth_k: bool = True, pv_mode: int = SAGE_PV_FP16,
             sm_scale: float = 0.0, out=None, stream=None, smooth_v: bool = False,
             fine: bool = False, smooth_q: bool = False):
    """O = SageAttention(q, k, v) for fp16 CUDA tensors q [B, H, Nq, d], k and v
    [B, H, Nk, d] (Nq != Nk: sage_attn_fwd_kv, causal mask aligned at the bottom right)."""
    import torch
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    _want_fp16(q, k, v)
    _want_size("k", k, B * H * Nk * d)
    _want_size("v", v, B * H * Nk * d)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want_out(out, q)
    flags = _smooth_flags(smooth_k, smooth_v, fine, smooth_q)
    if Nq == Nk:
        sage_attn_fwd(q, k, v, out, B, H, Nq, d, causal, flags, pv_mode, sm_scale, stream)
    else:
        sage_attn_fwd_kv(q, k, v, out, B, H, Nq, Nk, d, causal, flags, pv_mode, sm_scale, None, 0,
                         stream)
    return out


def sageattn_varlen_kv(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                       causal: bool = False, smooth_k: bool = True,
                       pv_mode: int = SAGE_PV_FP16, sm_scale: float = 0.0, out=None,
                       stream=None, smooth_v: bool = False, fine: bool = False,
                       smooth_q: bool = False):
    """Packed sequences with their own query and key lengths: q [Tq, H, d], k and v
    [Tk, H, d], cu_seqlens_q / cu_seqlens_k int32 [nseq+1] on the device. The options are
    sageattn's."""
    import torch
    Tq, H, d = q.shape
    Tk = k.shape[0]
    _want_fp16(q, k, v)
    _want_size("k", k, Tk * H * d)
    _want_size("v", v, Tk * H * d, k)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want_out(out, q)
    sage_attn_varlen_fwd_kv(q, k, v, out, cu_seqlens_q, cu_seqlens_k, cu_seqlens_q.numel() - 1,
                            Tq, Tk, max_seqlen_q, max_seqlen_k, H, d, causal,
                            _smooth_flags(smooth_k, smooth_v, fine, smooth_q), pv_mode, sm_scale,
                            None, 0, stream)
    return out


def sageattn_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False,
                    smooth_k: bool = True, pv_mode: int = SAGE_PV_FP16, sm_scale: float = 0.0,
                    out=None, stream=None, smooth_v: bool = False, fine: bool = False,
                    smooth_q: bool = False):
    """SageAttention over packed sequences: q, k, v [T, H, d], cu_seqlens int32 [nseq+1].
    The options are sageattn's."""
    import torch
    T, H, d = q.shape
    _want_fp16(q, k, v)
    _want_size("k", k, T * H * d, q)
    _want_size("v", v, T * H * d, q)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want_out(out, q)
    sage_attn_varlen_fwd(q, k, v, out, cu_seqlens, cu_seqlens.numel() - 1, T, max_seqlen, H, d,
                         causal, _smooth_flags(smooth_k, smooth_v, fine, smooth_q), pv_mode,
                         sm_scale, None, 0, stream)
    return out


def quant_qk(q, k, smooth_k: bool = True, stream=None, fine: bool = False,
             smooth_q: bool = False):
    """Dense smooth-K + INT8: dict of q_i8, q_scale, k_i8, k_scale, k_mean (q [B,H,Nq,d]
    and k [B,H,Nk,d] may differ in length; fine: per-token Q and per-32-token K scales;
    smooth_q: also q_mean [B,H,d] and the score compensation q_comp [B,H,ceil(Nk/128)*128])."""
    import torch
    B, H, N, d = q.shape
    Nk = k.shape[2]
    _want_fp16(q, k)
    _want_size("k", k, B * H * Nk * d)
    dev = q.device
    qg, kg = (1, 32) if fine else (Q_BLOCK, K_BLOCK)
    z = dict(q_i8=torch.empty(q.shape, dtype=torch.int8, device=dev),
             q_scale=torch.empty((B, H, math.ceil(N / qg)), dtype=torch.float32, device=dev),
             k_i8=torch.empty(k.shape, dtype=torch.int8, device=dev),
             k_scale=torch.empty((B, H, math.ceil(Nk / kg)), dtype=torch.float32, device=dev),
             k_mean=torch.empty((B, H, d), dtype=torch.float32, device=dev))
    flags = ((SAGE_SMOOTH_K if smooth_k else 0) | (SAGE_QK_FINE if fine else 0)
             | (SAGE_SMOOTH_Q if smooth_q else 0))
    if smooth_q:
        z["q_mean"] = torch.empty((B, H, d), dtype=torch.float32, device=dev)
        z["q_comp"] = torch.empty((B, H, math.ceil(Nk / 128) * 128), dtype=torch.float32,
                                  device=dev)
    if N == Nk and not fine and not smooth_q:
        sage_quant_qk(q, k, z["q_i8"], z["q_scale"], z["k_i8"], z["k_scale"], z["k_mean"], B, H, N,
                      d, smooth_k, stream)
    else:
        sage_quant_qk_kv(q, k, z["q_i8"], z["q_scale"], z["k_i8"], z["k_scale"], z["k_mean"],
                         z.get("q_mean"), z.get("q_comp"), B, H, N, Nk, d, flags, None, 0, stream)
    return z


def quant_qk_varlen(q, k, cu_seqlens, max_seqlen: int, smooth_k: bool = True, stream=None,
                    fine: bool = False):
    import torch
    T, H, d = q.shape
    nseq = cu_seqlens.numel() - 1
    _want_fp16(q, k)
    _want_size("k", k, T * H * d, q)
    dev = q.device
    qg, kg = (1, 32) if fine else (Q_BLOCK, K_BLOCK)
    z = dict(q_i8=torch.empty(q.shape, dtype=torch.int8, device=dev),
             q_scale=torch.empty((nseq, H, math.ceil(max_seqlen / qg)), dtype=torch.float32,
                                 device=dev),
             k_i8=torch.empty(k.shape, dtype=torch.int8, device=dev),
             k_scale=torch.empty((nseq, H, math.ceil(max_seqlen / kg)), dtype=torch.float32,
                                 device=dev),
             k_mean=torch.empty((nseq, H, d), dtype=torch.float32, device=dev))
    flags = (SAGE_SMOOTH_K if smooth_k else 0) | (SAGE_QK_FINE if fine else 0)
    sage_quant_qk_varlen(q, k, cu_seqlens, nseq, T, max_seqlen, H, d, z["q_i8"], z["q_scale"],
                         z["k_i8"], z["k_scale"], z["k_mean"], flags, stream)
    return z


def quant_v_fp8(v, stream=None, smooth_v: bool = False):
    """Dense V -> (E4M3 codes as uint8 [B,H,N,d], per-channel scales [B,H,d]); with
    smooth_v, a third result: the channel mean of V [B,H,d] the codes are taken from."""
    import torch
    B, H, N, d = v.shape
    _want_fp16(v)
    codes = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    scales = torch.empty((B, H, d), dtype=torch.float32, device=v.device)
    if not smooth_v:
        sage_quant_v_fp8(v, codes, scales, B, H, N, d, stream)
        return codes, scales
    mean = torch.empty((B, H, d), dtype=torch.float32, device=v.device)
    sage_quant_v_fp8_smooth(v, codes, scales, mean, B, H, N, d, stream)
    return codes, scales, mean


def quant_v_fp8_varlen(v, cu_seqlens, max_seqlen: int, stream=None, smooth_v: bool = False):
    import torch
    T, H, d = v.shape
    nseq = cu_seqlens.numel() - 1
    _want_fp16(v)
    codes = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    scales = torch.empty((nseq, H, d), dtype=torch.float32, device=v.device)
    if not smooth_v:
        sage_quant_v_fp8_varlen(v, cu_seqlens, nseq, T, max_seqlen, H, d, codes, scales, stream)
        return codes, scales
    mean = torch.empty((nseq, H, d), dtype=torch.float32, device=v.device)
    sage_quant_v_fp8_smooth_varlen(v, cu_seqlens, nseq, T, max_seqlen, H, d, codes, scales, mean,
                                   stream)
    return codes, scales, mean


def attn_quantized(q_i8, q_scale, k_i8, k_scale, v, v_scale, causal: bool = False,
                   pv_mode: int = SAGE_PV_FP16, sm_scale: float = 0.0, out=None, stream=None,
                   v_mean=None, fine: bool = False, q_comp=None):
    """Step 3 on pre-quantized operands; v_mean (FP8 mode) selects the smooth-V epilogue,
    fine the per-token Q / per-32-token K scale layout, q_comp the smooth-Q compensation."""
    import torch
    B, H, N, d = q_i8.shape
    Nk = k_i8.shape[2]
    if pv_mode == SAGE_PV_FP16:
        _want_fp16(v)
    if out is None:
        out = torch.empty(q_i8.shape, dtype=torch.float16, device=q_i8.device)
    if Nk != N or fine or q_comp is not None:
        sage_attn_fwd_quantized_kv(q_i8, q_scale, k_i8, k_scale, v, v_scale, v_mean, q_comp, out,
                                   B, H, N, Nk, d, causal, pv_mode, sm_scale,
                                   SAGE_QK_FINE if fine else 0, stream)
        return out
    if v_mean is not None:
        if pv_mode != SAGE_PV_FP8:
            raise ValueError("v_mean needs the FP8 P.V mode")
        sage_attn_fwd_quantized_smooth_v(q_i8, q_scale, k_i8, k_scale, v, v_scale, v_mean, out,
                                         B, H, N, d, causal, sm_scale, stream)
        return out
    sage_attn_fwd_quantized(q_i8, q_scale, k_i8, k_scale, v, v_scale, out, B, H, N, d, causal,
                            pv_mode, sm_scale, stream)
    return out


def attn_decode(q_i8, q_scale, k_i8, k_scale, v, causal: bool = False, sm_scale: float = 0.0,
                out=None, stream=None, fine: bool = False, workspace=None):
    """Step 3 for a few queries (Nq <= DECODE_MAX_Q) on pre-quantized operands, FP16 P.V,
    split over the keys (sage_attn_decode_quantized); the workspace is allocated here
    unless given."""
    import torch
    B, H, Nq, d = q_i8.shape
    Nk = k_i8.shape[2]
    _want_fp16(v)
    if out is None:
        out = torch.empty(q_i8.shape, dtype=torch.float16, device=q_i8.device)
    need = sage_attn_decode_workspace_size(B, H, Nq, Nk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q_i8.device)
    sage_attn_decode_quantized(q_i8, q_scale, k_i8, k_scale, v, out, B, H, Nq, Nk, d, causal,
                               sm_scale, SAGE_QK_FINE if fine else 0, workspace,
                               workspace.numel() * workspace.element_size(), stream)
    return out


# Rotary positions and the paged 4-bit cache. A decode step makes these calls once per layer and
# their kernels take a few microseconds, so the checks of shapes, types and devices, the outputs'
# allocation and the call itself are compiled (csrc/binding.cpp, built beside libsage.so): 4 to
# 6 us a call against 13 to 15 in Python. A wrong tensor raises ValueError there.

ROPE_SCALINGS = {"plain": SAGE_ROPE_PLAIN, "linear": SAGE_ROPE_LINEAR, "base": SAGE_ROPE_BASE,
                 "parts": SAGE_ROPE_PARTS}
_calls = None


def _bound():
    """The compiled binding, bound to the library's entry points; raises if it is missing."""
    global _calls
    import torch  # noqa: F401  (its libraries first)
    try:
        from . import _binding as b
    except ImportError as e:
        raise RuntimeError("quantized_attention_03_b200/_binding.so is missing or does not fit this torch: "
                           "build it with `python -m quantized_attention_03_b200.build`") from e
    from .build import binding_for
    if b.built_for != binding_for():
        raise RuntimeError(f"quantized_attention_03_b200/_binding.so is built for {b.built_for}, this is "
                           f"{binding_for()}: build it with `python -m quantized_attention_03_b200.build`")
    L = lib()
    b.bind(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
        "sage_rope", "sage_kv4_append", "sage_kv4_gather", "sage_attn_kv4", "sage_attn_kv4_workspace_size")))
    _calls = b
    return b


def _done(name: str, r):
    """What a compiled call returned, or the error it stands for."""
    if type(r) is int:
        raise SageError(name, r)
    return r


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
               device="cuda"):
    """Angles per position of the rot_dim/2 rotated pairs (float64 tensor) and the factor on
    cos and sin that belongs to them. scaling: "plain", "linear", "base" or "parts" (see
    sage_rope_freqs in sage.h)."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling is one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    freqs = torch.empty(max(rot_dim // 2, 0), dtype=torch.float64)
    mscale = (ctypes.c_double * 1)()
    sage_rope_freqs(freqs if rot_dim > 1 else None, mscale, rot_dim, base, ROPE_SCALINGS[scaling],
                    factor, original_len, beta_fast, beta_slow)
    return freqs.to(device), mscale[0]


def rope(q, k, freqs, positions=None, mscale: float = 1.0, interleaved: bool = False,
         inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [B, Hq, N, d] and k [B, Hk, N, d], or packed [T, H, d] (any
    strides; k may be None): (q_out, k_out). freqs and mscale: rope_freqs. positions int32 [N],
    [B, N] or [T]; None: 0 .. N-1. interleaved: pairs (2i, 2i+1), else (i, i + rot/2). inverse:
    by the negative angles, with the same mscale: the transpose of the rotation, which is its
    gradient (and at mscale 1 the way back). Autograd goes through the call: where q or k
    requires a gradient, so do the results, and q_out and k_out cannot be given. q_out=q,
    k_out=k rotates in place; outputs that overlap inputs or each other otherwise raise
    ValueError where that can be seen."""
    r = (_calls or _bound()).rope(q, k, freqs, positions, mscale, interleaved, inverse, q_out, k_out,
                                  None if stream is None else _stream(stream))
    if r == -1:
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out take no gradient")
        return _rope_autograd(q, k, freqs, positions, mscale, interleaved, inverse, stream)
    return _done("sage_rope", r)


_rope_function = None


def _rope_autograd(q, k, freqs, positions, mscale, interleaved, inverse, stream):
    """rope as a node of autograd's graph; its backward is rope again, with the other angles."""
    global _rope_function
    import torch
    if _rope_function is None:
        class Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, freqs, positions, mscale, interleaved, inverse):
                ctx.set_materialize_grads(False)
                ctx.save_for_backward(freqs, positions)
                ctx.how = mscale, interleaved, inverse
                out = rope(q, k, freqs, positions, mscale, interleaved, inverse)
                ctx.mark_non_differentiable(*(x for x, need in zip(out, ctx.needs_input_grad)
                                              if x is not None and not need))
                return out

            @staticmethod
            def backward(ctx, q, k):
                mscale, interleaved, inverse = ctx.how
                freqs, positions = ctx.saved_tensors
                # a gradient comes in whatever layout the graph gave it
                x = [g if g is None or (g.stride(-1) == 1 and all(s % 8 == 0 for s in g.stride()[:-1])
                                        and g.data_ptr() % 16 == 0)
                     else g.clone(memory_format=torch.contiguous_format)
                     for g in (g if need else None for g, need in zip((q, k), ctx.needs_input_grad))]
                if x[0] is not None:
                    x = rope(x[0], x[1], freqs, positions, mscale, interleaved, not inverse)
                elif x[1] is not None:
                    x = None, rope(x[1], None, freqs, positions, mscale, interleaved, not inverse)[0]
                return *x, None, None, None, None, None

        _rope_function = Rope
    args = q, k, freqs, positions, mscale, interleaved, inverse
    if stream is None:
        return _rope_function.apply(*args)
    raw = _stream(stream)                               # the backward pass runs on it too
    with torch.cuda.stream(torch.cuda.default_stream(q.device) if raw == 0
                           else torch.cuda.ExternalStream(raw, q.device)):
        return _rope_function.apply(*args)


def kv4_cache(num_pages: int, Hkv: int, page_size: int, d: int, device="cuda"):
    """An empty paged 4-bit cache for head dim d: uint8 [num_pages, Hkv, page bytes]."""
    import torch
    n = sage_kv4_page_bytes(page_size, d)
    if n == 0:
        raise ValueError(f"page_size is a power of two from 16 to 256 and d is 64 or 128, got {page_size} and {d}")
    return torch.empty((num_pages, Hkv, n), dtype=torch.uint8, device=device)


def kv4_append(cache, block_table, kv_lens, cu_seqlens, k, v, q=None, freqs=None,
               mscale: float = 1.0, interleaved: bool = False, k_mean=None, q_out=None,
               stream=None):
    """Writes new tokens' k and v [T, Hkv, d] (any token and head strides) into the paged 4-bit
    cache as the last tokens of their sequences, k rotated by their positions (freqs, mscale:
    rope_freqs; None: not rotated) and lessened by k_mean [Hkv, d]; returns q [T, Hq, d] rotated
    alike, or None; k_mean leaves attn_kv4's output as it is and its lse smaller. No gradient
    passes. kv_lens int32 [nseq] counts the new tokens, cu_seqlens int32 [nseq+1] says
    which rows are whose (None: T / nseq each), block_table int32 [nseq, max_pages] where the
    pages are."""
    return _done("sage_kv4_append", (_calls or _bound()).kv4_append(
        cache, block_table, kv_lens, cu_seqlens, k, v, q, freqs, mscale, interleaved, k_mean, q_out,
        None if stream is None else _stream(stream)))


def kv4_gather(cache, block_table, kv_lens, cu_seqlens, total: int, d: int, dtype=None,
               rep: int = 1, k_out=None, v_out=None, stream=None):
    """The last cu_seqlens[s+1] - cu_seqlens[s] tokens of every sequence as 16-bit k and v
    [total, Hkv * rep, d], each head rep times, d that of kv4_cache. In float16 (the default)
    they are what sageattn_varlen_kv takes, with float16 queries, for a prefill chunk over
    cached keys; this package's prefill attention takes no bfloat16."""
    import torch
    if dtype not in (None, torch.float16, torch.bfloat16):
        raise ValueError(f"dtype is float16 or bfloat16, got {dtype}")
    return _done("sage_kv4_gather", (_calls or _bound()).kv4_gather(
        cache, block_table, kv_lens, cu_seqlens, total, d, dtype is torch.bfloat16, rep, k_out, v_out,
        None if stream is None else _stream(stream)))


def attn_kv4(q, cache, block_table, kv_lens, cu_seqlens=None, max_q: Optional[int] = None,
             causal: bool = True, sm_scale: float = 0.0, out=None, lse=None, workspace=None,
             stream=None):
    """Attention of q [T, Hq, d] (any token and head strides) over the paged 4-bit cache; query
    head h reads key head h // (Hq / Hkv). A sequence has at most max_q queries, which are its
    last tokens (by default T / nseq without cu_seqlens, else DECODE_MAX_Q: give the least that
    holds, since one query a sequence takes 1.7 to 1.8 times as long with 16). lse: float32
    [T, Hq] that takes the log of the softmax sums, over keys as the cache holds them (lessened by
    k_mean). The workspace is allocated here unless given; what is allocated belongs to the stream
    that the call runs on. No gradient passes, as none does in the package's attention."""
    return _done("sage_attn_kv4", (_calls or _bound()).attn_kv4(
        q, cache, block_table, kv_lens, cu_seqlens, max_q, causal, sm_scale, out, lse, workspace,
        None if stream is None else _stream(stream)))


def qk_int32(q_i8, k_i8, stream=None):
    """Debug: the int32 score matrices S = q_i8 k_i8^T [B,H,N,N] from the tensor-core pass."""
    import torch
    B, H, N, d = q_i8.shape
    s = torch.zeros((B, H, N, N), dtype=torch.int32, device=q_i8.device)
    sage_debug_qk_int32(q_i8, k_i8, s, B, H, N, d, stream)
    return s
