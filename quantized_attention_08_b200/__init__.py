"""Python binding of libsage.so: SageAttention-style quantized attention on B200.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/sage.h.  PyTorch supplies device
memory and the current stream.  There is no fallback: if the library is not
built, or the GPU is not a B200, the calls raise.

Functions carry the names of the C entry points:
  sage_smooth_quant_qk, sage_smooth_quant_qk_noalloc, sage_quant_v_fp8,
  sage_smooth_quant_qkv, sage_smooth_quant_qkv_rope,
  sage_attn_fwd_quantized,
  sage_attn_fwd, sage_attn_fwd_ws, sage_attn_workspace_bytes,
  sage_attn_fwd_host, sage_smooth_quant_qkv_varlen, sage_attn_fwd_varlen_quantized,
  sage_attn_fwd_varlen, sage_get_device_error, sage_set_wait_timeout_ns,
  sage_selftest_wait_timeout, sage_status_string, sage_version,
  sage_v_hat_layout.
Serving from a paged key-value cache (SageKVCache holds one; fp16 and bf16):
  sage_kv_slots, sage_rope_axes, sage_kv_append, sage_attn_decode_paged,
  sage_attn_decode_workspace_bytes.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsage.so")

SAGE_OK = 0
SAGE_ERR_DEVICE_TIMEOUT = 6
VARIANTS = {"B": 0, "8+8": 1, "8+8-r56": 2}

_c = ctypes
_vp = _c.c_void_p
_i = _c.c_int
_f = _c.c_float

_SIGS = {
    "sage_smooth_quant_qk": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp]),
    "sage_smooth_quant_qk_noalloc": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp,
                                          _vp]),
    "sage_quant_v_fp8": (_i, [_vp, _i, _i, _i, _i, _f, _vp, _vp, _vp]),
    "sage_smooth_quant_qkv": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp]),
    "sage_smooth_quant_qkv_rope": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "sage_attn_fwd_quantized": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp]),
    "sage_attn_workspace_bytes": (_c.c_size_t, [_i, _i, _i, _i, _i, _i]),
    "sage_attn_fwd": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "sage_attn_fwd_ws": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _c.c_size_t, _vp]),
    "sage_attn_fwd_host": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "sage_smooth_quant_qkv_varlen": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _f, _vp,
                                          _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "sage_attn_fwd_varlen_quantized": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                            _i, _i, _i, _i, _vp]),
    "sage_attn_fwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                                  _vp]),
    "sage_kv_slots": (_i, [_vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp,
                           _vp]),
    "sage_rope_axes": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                            _i, _i, _i, _i, _vp]),
    "sage_kv_append": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp]),
    "sage_attn_decode_paged": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp,
                                    _c.c_size_t, _vp]),
    "sage_attn_decode_workspace_bytes": (_c.c_size_t, [_i, _i, _i, _i, _i, _i, _i]),
    "sage_v_hat_layout": (_i, []),
    "sage_get_device_error": (_i, [_vp, _c.POINTER(_c.c_uint32)]),
    "sage_set_wait_timeout_ns": (None, [_c.c_uint64]),
    "sage_selftest_wait_timeout": (_i, [_c.c_uint64, _vp]),
    "sage_status_string": (_c.c_char_p, [_i]),
    "sage_version": (_c.c_char_p, []),
    "sage_last_error_detail": (_c.c_char_p, []),
}

_lib_handle = None


def load_library() -> ctypes.CDLL:
    """Load libsage.so (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build the CUDA library first "
                "(python -m quantized_attention_08_b200.build)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib_handle = lib
    return _lib_handle


class SageError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {sage_status_string(status)} (status {status}); "
                         f"last failing step: {sage_last_error_detail()}")


def sage_last_error_detail() -> str:
    return load_library().sage_last_error_detail().decode()


def sage_status_string(status: int) -> str:
    return load_library().sage_status_string(int(status)).decode()


def sage_version() -> str:
    return load_library().sage_version().decode()


def sage_v_hat_layout() -> int:
    return load_library().sage_v_hat_layout()


def _check(status: int, where: str):
    if status != SAGE_OK:
        raise SageError(status, where)


def _stream(stream=None) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str, cuda: bool = True):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if cuda and not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _variant(v) -> int:
    return VARIANTS[v] if isinstance(v, str) else int(v)


def _nb(N: int) -> int:
    return (N + 127) // 128


def sage_smooth_quant_qk(q: torch.Tensor, k: torch.Tensor, sm_scale: Optional[float] = None,
                         out=None, stream=None):
    """Smooth K, quantize Q*sm_scale and smoothed K per 128-token block.
    Returns (q_hat int8, k_hat int8, delta_q fp32, delta_k fp32, mean_k fp32)."""
    _need(q, torch.float16, "q")
    _need(k, torch.float16, "k")
    B, H, N, d = q.shape
    Hk = k.shape[1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        dev = q.device
        out = (torch.empty_like(q, dtype=torch.int8), torch.empty_like(k, dtype=torch.int8),
               torch.empty(B, H, _nb(N), dtype=torch.float32, device=dev),
               torch.empty(B, Hk, _nb(N), dtype=torch.float32, device=dev),
               torch.empty(B, Hk, d, dtype=torch.float32, device=dev))
    qh, kh, dq, dk, mk = out
    st = load_library().sage_smooth_quant_qk(_ptr(q), _ptr(k), B, H, Hk, N, d, float(sm_scale),
                                             _ptr(qh), _ptr(kh), _ptr(dq), _ptr(dk), _ptr(mk),
                                             _stream(stream))
    _check(st, "sage_smooth_quant_qk")
    return out


def sage_smooth_quant_qk_noalloc(q: torch.Tensor, k: torch.Tensor, out,
                                 sm_scale: Optional[float] = None, stream=None):
    """sage_smooth_quant_qk with no device allocation inside the call: the
    caller passes the five output tensors `out` = (q_hat, k_hat, delta_q,
    delta_k, mean_k) and the library uses its static 4 MiB scratch (sizes
    with B*H_kv*ceil(N/256)*d > 524288 raise).  Calls that may overlap on
    one device race on that scratch; see include/sage.h."""
    _need(q, torch.float16, "q")
    _need(k, torch.float16, "k")
    B, H, N, d = q.shape
    Hk = k.shape[1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    qh, kh, dq, dk, mk = out
    st = load_library().sage_smooth_quant_qk_noalloc(
        _ptr(q), _ptr(k), B, H, Hk, N, d, float(sm_scale), _ptr(qh), _ptr(kh), _ptr(dq),
        _ptr(dk), _ptr(mk), _stream(stream))
    _check(st, "sage_smooth_quant_qk_noalloc")
    return out


def sage_quant_v_fp8(v: torch.Tensor, v_r: float = 448.0, out=None, stream=None):
    """E4M3 codes of V / delta_v with delta_v = colmax|V| / v_r per channel.
    Returns (v_hat uint8 [B,Hkv,N,d], delta_v fp32 [B,Hkv,d])."""
    _need(v, torch.float16, "v")
    B, Hk, N, d = v.shape
    if out is None:
        out = (torch.empty_like(v, dtype=torch.uint8),
               torch.empty(B, Hk, d, dtype=torch.float32, device=v.device))
    vh, dv = out
    st = load_library().sage_quant_v_fp8(_ptr(v), B, Hk, N, d, float(v_r), _ptr(vh), _ptr(dv),
                                         _stream(stream))
    _check(st, "sage_quant_v_fp8")
    return out


def sage_smooth_quant_qkv(q, k, v=None, sm_scale: Optional[float] = None, v_r: float = 448.0,
                          out=None, stream=None):
    """Whole pre-pass in three launches.  Returns (q_hat, k_hat, delta_q,
    delta_k, mean_k, v_hat, delta_v); the last two are None when v is None."""
    _need(q, torch.float16, "q")
    _need(k, torch.float16, "k")
    if v is not None:
        _need(v, torch.float16, "v")
    B, H, N, d = q.shape
    Hk = k.shape[1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        dev = q.device
        out = (torch.empty_like(q, dtype=torch.int8), torch.empty_like(k, dtype=torch.int8),
               torch.empty(B, H, _nb(N), dtype=torch.float32, device=dev),
               torch.empty(B, Hk, _nb(N), dtype=torch.float32, device=dev),
               torch.empty(B, Hk, d, dtype=torch.float32, device=dev),
               None if v is None else torch.empty_like(v, dtype=torch.uint8),
               None if v is None else torch.empty(B, Hk, d, dtype=torch.float32, device=dev))
    qh, kh, dq, dk, mk, vh, dv = out
    st = load_library().sage_smooth_quant_qkv(
        _ptr(q), _ptr(k), _ptr(v), B, H, Hk, N, d, float(sm_scale), float(v_r), _ptr(qh),
        _ptr(kh), _ptr(vh), _ptr(dq), _ptr(dk), _ptr(mk), _ptr(dv), _stream(stream))
    _check(st, "sage_smooth_quant_qkv")
    return out


def sage_smooth_quant_qkv_rope(q, k, cos_t, sin_t, v=None, sm_scale: Optional[float] = None,
                               v_r: float = 448.0, out=None, stream=None):
    """sage_smooth_quant_qkv with rotary embedding of Q and K fused in front
    of the quantizers; cos_t / sin_t are fp32 CUDA tensors [N, d/2].  Same
    outputs as sage_smooth_quant_qkv."""
    _need(q, torch.float16, "q")
    _need(k, torch.float16, "k")
    _need(cos_t, torch.float32, "cos_t")
    _need(sin_t, torch.float32, "sin_t")
    if v is not None:
        _need(v, torch.float16, "v")
    B, H, N, d = q.shape
    Hk = k.shape[1]
    if tuple(cos_t.shape) != (N, d // 2) or tuple(sin_t.shape) != (N, d // 2):
        raise ValueError(f"rotary tables must be [N, d/2] = [{N}, {d // 2}]")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if out is None:
        dev = q.device
        out = (torch.empty_like(q, dtype=torch.int8), torch.empty_like(k, dtype=torch.int8),
               torch.empty(B, H, _nb(N), dtype=torch.float32, device=dev),
               torch.empty(B, Hk, _nb(N), dtype=torch.float32, device=dev),
               torch.empty(B, Hk, d, dtype=torch.float32, device=dev),
               None if v is None else torch.empty_like(v, dtype=torch.uint8),
               None if v is None else torch.empty(B, Hk, d, dtype=torch.float32, device=dev))
    qh, kh, dq, dk, mk, vh, dv = out
    st = load_library().sage_smooth_quant_qkv_rope(
        _ptr(q), _ptr(k), _ptr(v), _ptr(cos_t), _ptr(sin_t), B, H, Hk, N, d, float(sm_scale),
        float(v_r), _ptr(qh), _ptr(kh), _ptr(vh), _ptr(dq), _ptr(dk), _ptr(mk), _ptr(dv),
        _stream(stream))
    _check(st, "sage_smooth_quant_qkv_rope")
    return out


def sage_attn_fwd_quantized(q_hat, k_hat, delta_q, delta_k, v_or_vhat, delta_v=None, *,
                            causal: bool = False, variant="B", o=None, stream=None):
    """Attention on pre-quantized operands; returns o fp16 [B,H,N,d]."""
    _need(q_hat, torch.int8, "q_hat")
    _need(k_hat, torch.int8, "k_hat")
    var = _variant(variant)
    B, H, N, d = q_hat.shape
    Hk = k_hat.shape[1]
    if o is None:
        o = torch.empty(B, H, N, d, dtype=torch.float16, device=q_hat.device)
    st = load_library().sage_attn_fwd_quantized(
        _ptr(q_hat), _ptr(k_hat), _ptr(delta_q), _ptr(delta_k), _ptr(v_or_vhat), _ptr(delta_v),
        _ptr(o), B, H, Hk, N, d, int(bool(causal)), var, _stream(stream))
    _check(st, "sage_attn_fwd_quantized")
    return o


def sage_attn_workspace_bytes(B: int, H: int, H_kv: int, N: int, d: int, variant="B") -> int:
    return load_library().sage_attn_workspace_bytes(B, H, H_kv, N, d, _variant(variant))


def sage_attn_fwd(q, k, v, *, causal: bool = False, sm_scale: Optional[float] = None,
                  variant="B", o=None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Whole SageAttention forward (Smooth K, quantize, attention); returns o fp16."""
    _need(q, torch.float16, "q")
    _need(k, torch.float16, "k")
    _need(v, torch.float16, "v")
    B, H, N, d = q.shape
    Hk = k.shape[1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    lib = load_library()
    if workspace is None:
        st = lib.sage_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, Hk, N, d, int(bool(causal)),
                               float(sm_scale), _variant(variant), _stream(stream))
        _check(st, "sage_attn_fwd")
    else:
        st = lib.sage_attn_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, H, Hk, N, d,
                                  int(bool(causal)), float(sm_scale), _variant(variant),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
        _check(st, "sage_attn_fwd_ws")
    return o


def sage_attn_fwd_ws(q, k, v, workspace: torch.Tensor, *, causal: bool = False,
                     sm_scale: Optional[float] = None, variant="B", o=None, stream=None):
    """sage_attn_fwd with the intermediates carved from a caller workspace
    (a CUDA tensor of at least sage_attn_workspace_bytes() bytes)."""
    if workspace is None:
        raise ValueError("workspace is required")
    return sage_attn_fwd(q, k, v, causal=causal, sm_scale=sm_scale, variant=variant, o=o,
                         workspace=workspace, stream=stream)


def sage_attn_fwd_host(q_host, k_host, v_host, o_host, *, causal: bool = False,
                       sm_scale: Optional[float] = None, variant="B", stream=None):
    """End-to-end call on host (CPU, ideally pinned) fp16 tensors; o_host is written."""
    for t, n in ((q_host, "q_host"), (k_host, "k_host"), (v_host, "v_host"), (o_host, "o_host")):
        _need(t, torch.float16, n, cuda=False)
        if t.is_cuda:
            raise TypeError(f"{n} must be a host tensor")
    B, H, N, d = q_host.shape
    Hk = k_host.shape[1]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    st = load_library().sage_attn_fwd_host(_ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(o_host),
                                           B, H, Hk, N, d, int(bool(causal)), float(sm_scale),
                                           _variant(variant), _stream(stream))
    _check(st, "sage_attn_fwd_host")
    return o_host


def _varlen_shape(q, k, cu_seqlens, max_seqlen):
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    H, T, d = q.shape
    Hk = k.shape[0]
    B = cu_seqlens.numel() - 1
    return B, H, Hk, T, d, int(max_seqlen)


def sage_smooth_quant_qkv_varlen(q, k, cu_seqlens, max_seqlen: int, v=None,
                                 sm_scale: Optional[float] = None, v_r: float = 448.0, stream=None):
    """Pre-pass of a packed batch (q [H,T,d], k/v [H_kv,T,d], cu_seqlens int32
    [B+1] on the device).  Returns (q_hat, k_hat, delta_q [B,H,nbm],
    delta_k [B,H_kv,nbm], mean_k [B,H_kv,d], v_hat, delta_v)."""
    _need(q, torch.float16, "q")
    _need(k, torch.float16, "k")
    B, H, Hk, T, d, ms = _varlen_shape(q, k, cu_seqlens, max_seqlen)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    dev = q.device
    nbm = _nb(ms)
    qh, kh = torch.empty_like(q, dtype=torch.int8), torch.empty_like(k, dtype=torch.int8)
    dq = torch.zeros(B, H, nbm, dtype=torch.float32, device=dev)
    dk = torch.zeros(B, Hk, nbm, dtype=torch.float32, device=dev)
    mk = torch.empty(B, Hk, d, dtype=torch.float32, device=dev)
    vh = None if v is None else torch.empty_like(v, dtype=torch.uint8)
    dv = None if v is None else torch.empty(B, Hk, d, dtype=torch.float32, device=dev)
    st = load_library().sage_smooth_quant_qkv_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, ms, T, H, Hk, d, float(sm_scale),
        float(v_r), _ptr(qh), _ptr(kh), _ptr(vh), _ptr(dq), _ptr(dk), _ptr(mk), _ptr(dv),
        _stream(stream))
    _check(st, "sage_smooth_quant_qkv_varlen")
    return qh, kh, dq, dk, mk, vh, dv


def sage_attn_fwd_varlen_quantized(q_hat, k_hat, delta_q, delta_k, v_or_vhat, delta_v,
                                   cu_seqlens, max_seqlen: int, *, causal: bool = False,
                                   variant="B", o=None, stream=None):
    """Attention of a packed batch on pre-quantized operands; returns o
    fp16 [H,T,d]."""
    _need(q_hat, torch.int8, "q_hat")
    _need(k_hat, torch.int8, "k_hat")
    var = _variant(variant)
    B, H, Hk, T, d, ms = _varlen_shape(q_hat, k_hat, cu_seqlens, max_seqlen)
    if o is None:
        o = torch.empty(H, T, d, dtype=torch.float16, device=q_hat.device)
    st = load_library().sage_attn_fwd_varlen_quantized(
        _ptr(q_hat), _ptr(k_hat), _ptr(delta_q), _ptr(delta_k), _ptr(v_or_vhat), _ptr(delta_v),
        _ptr(o), _ptr(cu_seqlens), B, ms, T, H, Hk, d, int(bool(causal)), var, _stream(stream))
    _check(st, "sage_attn_fwd_varlen_quantized")
    return o


def sage_attn_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, *, causal: bool = False,
                         sm_scale: Optional[float] = None, variant="B", o=None, stream=None):
    """Whole forward pass of a packed batch: q [H,T,d], k/v [H_kv,T,d] fp16,
    cu_seqlens int32 [B+1] on the device; returns o fp16 [H,T,d]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.float16, n)
    B, H, Hk, T, d, ms = _varlen_shape(q, k, cu_seqlens, max_seqlen)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    st = load_library().sage_attn_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(cu_seqlens), B, ms, T, H, Hk, d,
        int(bool(causal)), float(sm_scale), _variant(variant), _stream(stream))
    _check(st, "sage_attn_fwd_varlen")
    return o


# ------------------------------------------------- serving from a paged cache
KV_FORMATS = {"16": 0, "B": 1, "8+8": 2}
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_i64x3 = _c.c_int64 * 3
_i64x4 = _c.c_int64 * 4
_i64x14 = _c.c_int64 * 14


class _CacheStruct(_c.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("k_page_stride", _c.c_int64), ("v_page_stride", _c.c_int64),
                ("k_scale_page_stride", _c.c_int64), ("v_scale_page_stride", _c.c_int64),
                ("num_pages", _i), ("page_size", _i), ("H_kv", _i), ("d", _i), ("format", _i),
                ("dtype", _i)]


# The serving calls of a decode step take microseconds on the GPU, so their
# checks keep to cheap accessors: device numbers for devices, torch's raw
# stream lookup, each library function looked up once, and outputs made like a
# tensor that exists (a third of torch.empty's time).
def _strided(t: torch.Tensor, dtype, name: str, dev: int):
    """Checks of a strided argument (type, device number, last axis dense);
    returns its strides."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    st = t.stride()
    if not st or st[-1] != 1:
        raise ValueError(f"{name} must be dense along its last axis")
    return st


def _dense(t: torch.Tensor, dtype, name: str, dev: int, shape) -> int:
    """Checks of a contiguous argument (type, device number, shape); returns
    its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_fns = {}


def _call(name: str, dev: int, *args):
    """Calls the library with device `dev` current, on its current stream."""
    if dev < 0:
        raise TypeError(f"{name} takes CUDA tensors")
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise SageError(status, name)


def _with_stream(f, stream, t, *args, **kw):
    """f with `stream` current, so that the outputs and workspaces that torch
    hands out belong to it."""
    if not isinstance(stream, torch.cuda.Stream):
        ptr = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(ptr, t.device) if ptr else torch.cuda.default_stream(t.device)
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.stream(stream):
        return f(t, *args, **kw)


class SageKVCache:
    """A paged key-value cache: k and v [num_pages, H_kv, page_size, d], with
    dense pages, and fp32 scales [num_pages, H_kv, page_size].  The format
    follows from the types: "16" (k and v fp16 or bf16), "B" (k int8 with
    k_scale, v 16-bit), "8+8" (k int8, v uint8 E4M3 codes, both scales; `dtype`
    is that of the model, fp16 unless given).  The tensors are the caller's
    and are used in place."""

    def __init__(self, k, v, k_scale=None, v_scale=None, dtype: Optional[torch.dtype] = None):
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must both be [num_pages, H_kv, page_size, d]")
        if k.dtype in _DTYPES and v.dtype == k.dtype:
            self.format, model = "16", k.dtype
        elif k.dtype == torch.int8 and v.dtype in _DTYPES:
            self.format, model = "B", v.dtype
        elif k.dtype == torch.int8 and v.dtype == torch.uint8:
            self.format, model = "8+8", dtype or torch.float16
        else:
            raise TypeError(f"no cache format has k {k.dtype} and v {v.dtype}")
        if model not in _DTYPES or (dtype is not None and dtype != model):
            raise TypeError(f"dtype {dtype} does not fit k {k.dtype} and v {v.dtype}")
        if not k.is_cuda:
            raise TypeError("k must be a CUDA tensor")
        self._dev = k.get_device()
        self.k, self.v, self.dtype, self.device = k, v, model, k.device
        self.k_scale = k_scale if self.format != "16" else None
        self.v_scale = v_scale if self.format == "8+8" else None
        self.num_pages, self.H_kv, self.page_size, self.d = k.shape
        s = self._struct = _CacheStruct()
        for name, t, inner in (("k", k, k.shape[1:]), ("v", v, k.shape[1:]),
                               ("k_scale", self.k_scale, k.shape[1:3]),
                               ("v_scale", self.v_scale, k.shape[1:3])):
            if t is None:
                if (name == "k_scale" and self.format != "16") or (name == "v_scale" and self.format == "8+8"):
                    raise ValueError(f"a cache of format {self.format} needs {name}")
                continue
            if name.endswith("scale"):
                if t.dtype != torch.float32 or t.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be fp32 [num_pages, H_kv, page_size]")
            if t.device != self.device:
                raise ValueError(f"{name} must be on {self.device}")
            if self.num_pages and not t[0].is_contiguous():
                raise ValueError(f"a page of {name} must be contiguous")
            n = 1
            for x in inner:
                n *= x
            setattr(s, name, t.data_ptr())
            setattr(s, name + "_page_stride", t.stride(0) if self.num_pages > 1 else n)
        s.num_pages, s.H_kv, s.page_size, s.d = k.shape
        s.format, s.dtype = KV_FORMATS[self.format], _DTYPES[model]
        self._ref = _c.addressof(s)

    @classmethod
    def allocate(cls, num_pages: int, H_kv: int, page_size: int, d: int, format: str = "8+8",
                 dtype: torch.dtype = torch.float16, device="cuda"):
        """A cache of zeros."""
        if format not in KV_FORMATS:
            raise ValueError(f"format must be one of {list(KV_FORMATS)}, got {format!r}")
        shape = (num_pages, H_kv, page_size, d)
        kt = dtype if format == "16" else torch.int8
        vt = torch.uint8 if format == "8+8" else dtype
        scale = lambda: torch.zeros(shape[:3], dtype=torch.float32, device=device)  # noqa: E731
        return cls(torch.zeros(shape, dtype=kt, device=device), torch.zeros(shape, dtype=vt, device=device),
                   scale() if format != "16" else None, scale() if format == "8+8" else None, dtype)


def sage_kv_slots(ctx_lens, new_lens, free_pages, free_used, block_table, *, page_size: int, T: int,
                  out=None, stream=None):
    """Block tables and slot maps of one step: ctx_lens, new_lens int32 [B],
    free_pages int32 [F] of which the first free_used (int32 [1]) are taken,
    block_table int32 [B, max_pages] (extended in place).  Returns (seq_lens
    [B], cu_seqlens [B+1], slot_map [T], positions [T], seq_ids [T],
    free_used [1]), all int32; `out` takes the same six tensors, of which
    seq_lens may be ctx_lens and free_used its input."""
    if stream is not None:
        return _with_stream(sage_kv_slots, stream, ctx_lens, new_lens, free_pages, free_used, block_table,
                            page_size=page_size, T=T, out=out)
    i32, dev = torch.int32, ctx_lens.get_device()
    B, F, width = ctx_lens.numel(), free_pages.numel(), block_table.shape[-1]
    if out is None:
        if T < 0 or page_size > 0x7fffffff:
            raise ValueError(f"T must not be negative, nor page_size past 2^31: got {T}, {page_size}")
        out = torch.empty(2 * B + 3 * T + 2, dtype=i32, device=ctx_lens.device).split_with_sizes(
            (B, B + 1, T, T, T, 1))
        lens = out[0].data_ptr()
        cu = lens + 4 * B
        slots = cu + 4 * B + 4
        pos, ids, used = slots + 4 * T, slots + 8 * T, slots + 12 * T
    else:
        lens, cu, slots, pos, ids, used = (
            _dense(t, i32, name, dev, (n,)) for t, name, n in
            zip(out, ("seq_lens", "cu_seqlens", "slot_map", "positions", "seq_ids", "free_used"),
                (B, B + 1, T, T, T, 1)))
    _call("sage_kv_slots", dev, _dense(ctx_lens, i32, "ctx_lens", dev, (B,)),
          _dense(new_lens, i32, "new_lens", dev, (B,)), B, _dense(free_pages, i32, "free_pages", dev, (F,)), F,
          _dense(free_used, i32, "free_used", dev, (1,)),
          _dense(block_table, i32, "block_table", dev, (B, width)), width, page_size, lens, cu, slots, pos, ids, T, used)
    return out


def sage_rope_axes(q, k, positions, inv_freq, sections, *, pairing: str = "half", q_out=None, k_out=None,
                   stream=None):
    """Rotary positions with several axes of q [B, H, N, d] and k [B, H_kv, N, d]
    (or [H, N, d] of one sequence; k may be None), any strides with a dense
    last axis.  positions int32 [axes, B, N] or [axes, N] (shared by the batch);
    sections: rotation pairs of each axis; inv_freq fp32 [sum(sections)];
    pairing "half" (i, i + R) or "interleaved" (2i, 2i + 1).  Returns (q, k)
    rotated, laid out as torch.empty_like lays them out; q_out / k_out take
    them instead (they may be q and k)."""
    if stream is not None:
        return _with_stream(sage_rope_axes, stream, q, k, positions, inv_freq, sections, pairing=pairing, q_out=q_out,
                            k_out=k_out)
    dtype, dev, shape = q.dtype, q.get_device(), q.shape
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"q must be torch.float16 or torch.bfloat16, got {dtype}")
    if pairing != "half" and pairing != "interleaved":
        raise ValueError(f"pairing must be 'half' or 'interleaved', got {pairing!r}")
    if len(shape) == 4:
        B, H, N, d = shape
    elif len(shape) == 3:
        B, (H, N, d) = 1, shape
    else:
        raise ValueError("q must be [B, H, N, d] or [H, N, d]")

    # strides of q, q_out, k, k_out (batch, head, token) and positions, in one array
    lead = () if len(shape) == 4 else (0,)
    if q_out is None:
        q_out = torch.empty_like(q)
    elif q_out.shape != shape:
        raise ValueError("q_out does not have the shape of its input")
    st = (*lead, *_strided(q, dtype, "q", dev)[:-1], *lead, *_strided(q_out, dtype, "q_out", dev)[:-1])
    if k is not None:
        kshape = k.shape
        if len(kshape) != len(shape) or kshape[-2:] != shape[-2:] or (not lead and kshape[0] != B):
            raise ValueError("q and k must have the same batch, tokens and channels")
        if k_out is None:
            k_out = torch.empty_like(k)
        elif k_out.shape != kshape:
            raise ValueError("k_out does not have the shape of its input")
        st += (*lead, *_strided(k, dtype, "k", dev)[:-1], *lead, *_strided(k_out, dtype, "k_out", dev)[:-1])
        Hk, kp, kop = kshape[-3], k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        Hk, kp, kop = 0, None, None
        st += (0,) * 6
    A = len(sections)
    ps = _strided(positions, torch.int32, "positions", dev)
    pshape = positions.shape
    if pshape == (A, B, N):
        st += ps[:2]
    elif pshape == (A, N):
        st += (ps[0], 0)
    else:
        raise ValueError(f"positions must be [{A}, {N}] or [{A}, {B}, {N}], got {tuple(pshape)}")
    inv = _dense(inv_freq, torch.float32, "inv_freq", dev, (sum(sections),))
    arr = _i64x14(*st)
    at = _c.addressof(arr)
    _call("sage_rope_axes", dev, q.data_ptr(), at, q_out.data_ptr(), at + 24, kp, at + 48, kop, at + 72,
          positions.data_ptr(), at + 96, inv, _axes(tuple(sections)), A, B, H, Hk, N, d, pairing != "half", code)
    return q_out, k_out


@functools.lru_cache(maxsize=64)
def _axes(sections):
    return (_i * len(sections))(*sections)


def sage_kv_append(k, v, slot_map, cache: SageKVCache, *, mean_k=None, seq_ids=None, stream=None):
    """Writes new K and V [H_kv, T, d] (any strides with a dense last axis) into
    the cache's slots slot_map int32 [T] (-1: skipped), quantized as the cache
    holds them.  mean_k fp32 [B, H_kv, d] with seq_ids int32 [T]: subtracted
    from K (Smooth K per request; every token of a request needs the same)."""
    if stream is not None:
        return _with_stream(sage_kv_append, stream, k, v, slot_map, cache, mean_k=mean_k, seq_ids=seq_ids)
    dev, shape = cache._dev, k.shape
    ks, vs = _strided(k, cache.dtype, "k", dev), _strided(v, cache.dtype, "v", dev)
    if len(shape) != 3 or v.shape != shape or shape[0] != cache.H_kv or shape[2] != cache.d:
        raise ValueError(f"k and v must both be [{cache.H_kv}, T, {cache.d}]")
    T = shape[1]
    B, mean, ids = 0, None, None
    if mean_k is not None:
        if seq_ids is None:
            raise ValueError("mean_k needs seq_ids")
        B = mean_k.shape[0]
        mean = _dense(mean_k, torch.float32, "mean_k", dev, (B, cache.H_kv, cache.d))
        ids = _dense(seq_ids, torch.int32, "seq_ids", dev, (T,))
    arr = _i64x4(ks[0], ks[1], vs[0], vs[1])
    at = _c.addressof(arr)
    _call("sage_kv_append", dev, k.data_ptr(), at, v.data_ptr(), at + 16, T,
          _dense(slot_map, torch.int32, "slot_map", dev, (T,)), mean, ids, B, cache._ref)
    return cache


def sage_attn_decode_workspace_bytes(B: int, H: int, H_kv: int, n_q: int, d: int, max_len: int,
                                     format="8+8") -> int:
    return load_library().sage_attn_decode_workspace_bytes(
        B, H, H_kv, n_q, d, max_len, KV_FORMATS[format] if isinstance(format, str) else int(format))


@functools.lru_cache(maxsize=1024)
def _decode_workspace(*sizes) -> int:
    return load_library().sage_attn_decode_workspace_bytes(*sizes)


def sage_attn_decode_paged(q, cache: SageKVCache, block_table, seq_lens, max_len: int, *,
                           causal: bool = True, sm_scale: Optional[float] = None, o=None,
                           return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of new tokens over the paged cache: q [B, H, n_q, d], or
    [B, H, d] of one token, any strides with a dense last axis; block_table
    int32 [B, max_pages], seq_lens int32 [B] (the new tokens included), max_len
    a bound on them.  causal: query i sees the keys up to its own token (the
    last n_q are the new ones).  Returns o (dense, q's shape), or (o, lse fp32)
    with return_lse.  workspace: a tensor of at least
    sage_attn_decode_workspace_bytes() bytes; taken from torch if not given."""
    if stream is not None:
        return _with_stream(sage_attn_decode_paged, stream, q, cache, block_table, seq_lens, max_len, causal=causal,
                            sm_scale=sm_scale, o=o, return_lse=return_lse, workspace=workspace)
    dev, d, shape = cache._dev, cache.d, q.shape
    qs = _strided(q, cache.dtype, "q", dev)
    if len(shape) == 4 and shape[3] == d:
        B, H, n_q, _ = shape
        arr = _i64x3(qs[0], qs[1], qs[2])
    elif len(shape) == 3 and shape[2] == d:
        B, H, _ = shape
        n_q = 1
        arr = _i64x3(qs[0], qs[1], 0)
    else:
        raise ValueError(f"q must be [B, H, n_q, {d}] or [B, H, {d}]")
    width = block_table.shape[-1]
    if max_len > 0x7fffffff:  # would wrap around in the C call
        raise ValueError(f"max_len must be below 2^31, got {max_len}")
    if o is None:
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = o.data_ptr()
    else:
        op = _dense(o, q.dtype, "o", dev, shape)
    lse, lp = None, None
    if return_lse:
        lse = torch.empty(shape[:-1], dtype=torch.float32, device=q.device)
        lp = lse.data_ptr()
    if workspace is None:
        size = _decode_workspace(B, H, cache.H_kv, n_q, d, max_len, cache._struct.format)
        ws = None
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    else:
        ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call("sage_attn_decode_paged", dev, q.data_ptr(), arr, cache._ref,
          _dense(block_table, torch.int32, "block_table", dev, (B, width)), width,
          _dense(seq_lens, torch.int32, "seq_lens", dev, (B,)), B, H, n_q, max_len, 1 if causal else 0,
          1.0 / math.sqrt(d) if sm_scale is None else sm_scale, op, lp, ws, size)
    return (o, lse) if return_lse else o


def sage_get_device_error(stream=None):
    """(status, raw error word); synchronizes the stream and clears the word."""
    w = ctypes.c_uint32(0)
    st = load_library().sage_get_device_error(_stream(stream), ctypes.byref(w))
    return st, w.value


def sage_set_wait_timeout_ns(ns: int):
    load_library().sage_set_wait_timeout_ns(int(ns))


def sage_selftest_wait_timeout(timeout_ns: int, stream=None):
    _check(load_library().sage_selftest_wait_timeout(int(timeout_ns), _stream(stream)),
           "sage_selftest_wait_timeout")
