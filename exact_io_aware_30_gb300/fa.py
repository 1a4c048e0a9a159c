"""ctypes binding of libfa.so (include/fa.h) -- argument marshalling only.

Every step of the attention forward, backward and paged decoding, of rotary
positions and of the paged cache's updates, writes and reads runs inside the library's CUDA
kernels; this module checks tensor metadata, allocates
outputs (and workspaces) with torch and passes raw pointers and sizes through
the C ABI.  If the library is missing or
refuses a request, it raises: there is no other code path.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import math
import os
import threading

from . import build as _build

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_CUDA = 4
FA_ERR_DEVICE_TIMEOUT = 5

MASK_NONE = 0
MASK_CAUSAL = 1
MASK_SLIDING_WINDOW = 2
MASKS = {"none": MASK_NONE, "causal": MASK_CAUSAL, "window": MASK_SLIDING_WINDOW,
         "sliding_window": MASK_SLIDING_WINDOW}

DTYPE_BF16 = 0
DTYPE_FP16 = 1
DTYPE_FP32 = 2             # fa_rope only
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
ROPE_FORWARD = 0
ROPE_BACKWARD = 1
PAGED_OK = 0               # per-request status of fa_paged_update
PAGED_NO_BLOCKS = 1
PAGED_TOO_LONG = 2
PAGED_NO_ROWS = 3
DECODE_AUTO = 0            # fa_decode_paged kernel choice
DECODE_TENSOR_CORES = 1
DECODE_CUDA_CORES = 2
_DECODE_KERNELS = {"auto": DECODE_AUTO, "tensor_cores": DECODE_TENSOR_CORES,
                   "cuda_cores": DECODE_CUDA_CORES}

# Every entry point declared in include/fa.h.
EXPORTS = ("fa_fwd", "fa_fwd_fp16", "fa_fwd_gqa", "fa_fwd_fp8", "fa_bwd", "fa_bwd_noalloc",
           "fa_bwd_workspace_query", "fa_decode_paged", "fa_decode_workspace_query",
           "fa_workspace_query", "fa_status_string", "fa_describe", "fa_get_device_error",
           "fa_fwd_host", "fa_fwd_host_workspace_query", "fa_set_debug_stall_ms",
           "fa_rope", "fa_rope_frequencies", "fa_paged_update", "fa_paged_update_by_request",
           "fa_cache_append_fp8",
           "fa_decode_paged_fp8", "fa_decode_fp8_workspace_query",
           "fa_cache_append_int4", "fa_cache_read_int4", "fa_decode_paged_int4",
           "fa_decode_int4_workspace_query")


class FAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None
_lock = threading.Lock()

_vp = ctypes.c_void_p
_i = ctypes.c_int


def lib_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load libfa.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB_PATH
        if not os.path.exists(p):
            raise FAError(-1, f"{p} is missing: build it with exact_io_aware_30_gb300.build.build()")
        lib = ctypes.CDLL(p)
        fwd_args = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _vp]
        for name in ("fa_fwd", "fa_fwd_fp16"):
            fn = getattr(lib, name)
            fn.restype = _i
            fn.argtypes = fwd_args
        lib.fa_fwd_gqa.restype = _i
        lib.fa_fwd_gqa.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                   ctypes.c_float, _i, _i, _i, _vp]
        lib.fa_bwd.restype = _i
        lib.fa_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                               _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _i, _vp]
        lib.fa_bwd_noalloc.restype = _i
        lib.fa_bwd_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _i, _vp]
        lib.fa_fwd_fp8.restype = _i
        lib.fa_fwd_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float,
                                   ctypes.c_float, ctypes.c_float, ctypes.c_float, _i, _i, _vp]
        lib.fa_decode_paged.restype = _i
        lib.fa_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                        _i, _i, _i, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i,
                                        _i, _i, _vp]
        lib.fa_decode_workspace_query.restype = _i
        lib.fa_decode_workspace_query.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                                  ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_set_debug_stall_ms.restype = _i
        lib.fa_set_debug_stall_ms.argtypes = [_i]
        lib.fa_bwd_workspace_query.restype = _i
        lib.fa_bwd_workspace_query.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i, _i,
                                               ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_fwd_host.restype = _i
        lib.fa_fwd_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i,
                                    _i, _i, _i, ctypes.c_float, _i, _i, _i, _vp]
        lib.fa_fwd_host_workspace_query.restype = _i
        lib.fa_fwd_host_workspace_query.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i, _i,
                                                    ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_workspace_query.restype = _i
        lib.fa_workspace_query.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i,
                                           ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_status_string.argtypes = [_i]
        _ll = ctypes.c_longlong
        lib.fa_rope.restype = _i
        lib.fa_rope.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ll, _ll, _vp,
                                ctypes.c_float, _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp]
        lib.fa_rope_frequencies.restype = _i
        lib.fa_rope_frequencies.argtypes = [_i, ctypes.c_double, _i, ctypes.c_double,
                                            ctypes.c_double, ctypes.c_double, ctypes.c_double, _vp,
                                            ctypes.POINTER(ctypes.c_float)]
        for name in ("fa_paged_update", "fa_paged_update_by_request"):
            fn = getattr(lib, name)
            fn.restype = _i
            fn.argtypes = [_vp] * 10 + [_i] * 5 + [_vp]
        lib.fa_cache_append_fp8.restype = _i
        lib.fa_cache_append_fp8.argtypes = [_vp, _vp, _ll, _ll, _ll, _ll, _vp, _vp, _vp, _vp, _vp,
                                            _i, _i, _i, _i, _i, _i, _vp]
        lib.fa_decode_paged_fp8.restype = _i
        lib.fa_decode_paged_fp8.argtypes = [_vp] * 10 + [ctypes.c_size_t] + [_i] * 9 + \
            [ctypes.c_float, _i, _i, _vp]
        lib.fa_decode_fp8_workspace_query.restype = _i
        lib.fa_decode_fp8_workspace_query.argtypes = [_i] * 11 + [ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_cache_append_int4.restype = _i
        lib.fa_cache_append_int4.argtypes = [_vp, _vp, _ll, _ll, _ll, _ll] + [_vp] * 5 + [_i] * 7 + [_vp]
        lib.fa_cache_read_int4.restype = _i
        lib.fa_cache_read_int4.argtypes = [_vp] * 11 + [_i] * 9 + [_vp]
        lib.fa_decode_paged_int4.restype = _i
        lib.fa_decode_paged_int4.argtypes = [_vp] * 10 + [ctypes.c_size_t] + [_i] * 10 + \
            [ctypes.c_float, _i, _i, _vp]
        lib.fa_decode_int4_workspace_query.restype = _i
        lib.fa_decode_int4_workspace_query.argtypes = [_i] * 12 + [ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_describe.restype = _i
        lib.fa_describe.argtypes = [_i, _i, _i, ctypes.c_char_p, ctypes.c_size_t]
        lib.fa_get_device_error.restype = _i
        lib.fa_get_device_error.argtypes = []
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != FA_OK:
        raise FAError(status, f"{what}: {status_string(status)}")


def mask_code(mask) -> int:
    return MASKS[mask] if isinstance(mask, str) else int(mask)


def fwd_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int, H: int,
            Sq: int, Sk: int, d: int, scale: float, mask_kind: int, window: int,
            stream: int, dtype: int = DTYPE_BF16) -> int:
    """Call fa_fwd / fa_fwd_fp16 with raw device pointers; returns the status."""
    lib = load()
    fn = lib.fa_fwd if dtype == DTYPE_BF16 else lib.fa_fwd_fp16
    return fn(_vp(q_ptr), _vp(k_ptr), _vp(v_ptr), _vp(o_ptr), _vp(lse_ptr), int(B), int(H),
              int(Sq), int(Sk), int(d), ctypes.c_float(scale), int(mask_kind), int(window),
              _vp(stream))


def fwd_gqa_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int, H: int,
                H_kv: int, Sq: int, Sk: int, d: int, scale: float, mask_kind: int, window: int,
                stream: int, dtype: int = DTYPE_BF16) -> int:
    """Call fa_fwd_gqa (K/V with H_kv heads) with raw device pointers; returns the status."""
    return load().fa_fwd_gqa(_vp(q_ptr), _vp(k_ptr), _vp(v_ptr), _vp(o_ptr), _vp(lse_ptr),
                             int(B), int(H), int(H_kv), int(Sq), int(Sk), int(d),
                             ctypes.c_float(scale), int(mask_kind), int(window), int(dtype),
                             _vp(stream))


def bwd_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, do_ptr: int,
            dq_ptr: int, dk_ptr: int, dv_ptr: int, ws_ptr: int, ws_bytes: int, B: int, H: int,
            H_kv: int, Sq: int, Sk: int, d: int, scale: float, mask_kind: int, window: int,
            stream: int, dtype: int = DTYPE_BF16) -> int:
    """Call fa_bwd with raw device pointers; returns the status."""
    return load().fa_bwd(_vp(q_ptr), _vp(k_ptr), _vp(v_ptr), _vp(o_ptr), _vp(lse_ptr),
                         _vp(do_ptr), _vp(dq_ptr), _vp(dk_ptr), _vp(dv_ptr), _vp(ws_ptr),
                         ctypes.c_size_t(ws_bytes), int(B), int(H), int(H_kv), int(Sq), int(Sk),
                         int(d), ctypes.c_float(scale), int(mask_kind), int(window), int(dtype),
                         _vp(stream))


def bwd_noalloc_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, do_ptr: int,
                    dq_ptr: int, dk_ptr: int, dv_ptr: int, B: int, H: int, H_kv: int, Sq: int,
                    Sk: int, d: int, scale: float, mask_kind: int, window: int, stream: int,
                    dtype: int = DTYPE_BF16) -> int:
    """Call fa_bwd_noalloc (the library's fixed workspace) with raw device pointers."""
    return load().fa_bwd_noalloc(_vp(q_ptr), _vp(k_ptr), _vp(v_ptr), _vp(o_ptr), _vp(lse_ptr),
                                 _vp(do_ptr), _vp(dq_ptr), _vp(dk_ptr), _vp(dv_ptr), int(B),
                                 int(H), int(H_kv), int(Sq), int(Sk), int(d),
                                 ctypes.c_float(scale), int(mask_kind), int(window), int(dtype),
                                 _vp(stream))


def fwd_fp8_raw(q_ptr, k_ptr, vt_ptr, o_ptr, lse_ptr, B, H, H_kv, Sq, Sk, d, scale, q_descale,
                k_descale, v_descale, mask_kind, window, stream) -> int:
    """Call fa_fwd_fp8 with raw device pointers; returns the status."""
    return load().fa_fwd_fp8(_vp(q_ptr), _vp(k_ptr), _vp(vt_ptr), _vp(o_ptr), _vp(lse_ptr), int(B),
                             int(H), int(H_kv), int(Sq), int(Sk), int(d), ctypes.c_float(scale),
                             ctypes.c_float(q_descale), ctypes.c_float(k_descale),
                             ctypes.c_float(v_descale), int(mask_kind), int(window), _vp(stream))


def forward_fp8(q, k, vt, q_descale: float, k_descale: float, v_descale: float,
                scale: float | None = None, mask="none", window: int = 0, out=None, lse=None,
                stream=None):
    """8-bit forward (fa_fwd_fp8) on CUDA uint8 tensors of e4m3 codes.

    q [B, H, Sq, d]; k [B, H_kv, Sk, d]; vt = V transposed [B, H_kv, d, Sk].
    Returns (o bf16 [B, H, Sq, d], lse fp32 [B, H, Sq]).
    """
    import torch
    for name, t in (("q", q), ("k", k), ("vt", vt)):
        if not t.is_cuda or not t.is_contiguous() or t.dim() != 4 or t.element_size() != 1:
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 4-D CUDA tensor of bytes")
    B, H, Sq, d = q.shape
    H_kv, Sk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, H_kv, Sk, d) or tuple(vt.shape) != (B, H_kv, d, Sk):
        raise FAError(FA_ERR_INVALID_ARG, "k must be [B,H_kv,Sk,d] and vt [B,H_kv,d,Sk]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, H, Sq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sp = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = fwd_fp8_raw(q.data_ptr(), k.data_ptr(), vt.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H,
                     H_kv, Sq, Sk, d, float(scale), float(q_descale), float(k_descale),
                     float(v_descale), mask_code(mask), int(window), sp)
    _check(st, "fa_fwd_fp8")
    return out, lse


def decode_raw(q_ptr, k_ptr, v_ptr, table_ptr, lens_ptr, o_ptr, lse_ptr, ws_ptr, ws_bytes, B, H,
               H_kv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len, scale, mask_kind,
               dtype, stream, kernel=DECODE_AUTO) -> int:
    """Call fa_decode_paged with raw device pointers; returns the status."""
    return load().fa_decode_paged(_vp(q_ptr), _vp(k_ptr), _vp(v_ptr), _vp(table_ptr),
                                  _vp(lens_ptr), _vp(o_ptr), _vp(lse_ptr), _vp(ws_ptr),
                                  ctypes.c_size_t(ws_bytes), int(B), int(H), int(H_kv), int(Sq),
                                  int(d), int(block_size), int(max_blocks), int(num_blocks),
                                  int(max_seq_len), ctypes.c_float(scale), int(mask_kind),
                                  int(dtype), int(kernel), _vp(stream))


def decode_kernel_code(kernel) -> int:
    """"auto", "tensor_cores", "cuda_cores" (or the FA_DECODE_* code)."""
    if isinstance(kernel, str):
        if kernel not in _DECODE_KERNELS:
            raise FAError(FA_ERR_UNSUPPORTED, f"decode kernel {kernel!r}: one of {list(_DECODE_KERNELS)}")
        return _DECODE_KERNELS[kernel]
    return int(kernel)


def decode_workspace_query(B, H, H_kv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len,
                           mask="none", dtype=DTYPE_BF16, kernel=DECODE_AUTO):
    """(status, bytes) of fa_decode_workspace_query."""
    n = ctypes.c_size_t(12345)
    st = load().fa_decode_workspace_query(int(B), int(H), int(H_kv), int(Sq), int(d),
                                          int(block_size), int(max_blocks), int(num_blocks),
                                          int(max_seq_len), mask_code(mask), int(dtype),
                                          decode_kernel_code(kernel), ctypes.byref(n))
    return st, n.value


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, max_seq_len: int,
                 scale: float | None = None, mask="none", out=None, lse=None, workspace=None,
                 stream=None, kernel="auto"):
    """Attention of q's new rows over a paged K/V cache (fa_decode_paged).

    q [B, H, Sq, d]; k_cache, v_cache [num_blocks, H_kv, block_size, d] (one
    16-bit dtype); block_table int32 [B, max_blocks] and seq_lens int32 [B] on
    the same CUDA device.  kernel: "auto" (the library's choice by rows per
    K/V head), "tensor_cores" or "cuda_cores".  Returns (o, lse).
    """
    import torch
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                    ("block_table", block_table), ("seq_lens", seq_lens)):
        if not t.is_cuda or not t.is_contiguous():
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous CUDA tensor")
    if not (q.dtype == k_cache.dtype == v_cache.dtype):
        raise FAError(FA_ERR_INVALID_ARG, "q and the caches must share one dtype")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise FAError(FA_ERR_INVALID_ARG, "block_table and seq_lens must be int32")
    dt = _dtype_code(q)
    B, H, Sq, d = q.shape
    nb, H_kv, bs, d2 = k_cache.shape
    if (tuple(v_cache.shape) != tuple(k_cache.shape) or d2 != d or block_table.dim() != 2
            or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,)):
        raise FAError(FA_ERR_INVALID_ARG, "shapes: q [B,H,Sq,d]; caches [blocks,H_kv,bs,d]; "
                      "block_table [B,n]; seq_lens [B]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    mb = block_table.shape[1]
    kc = decode_kernel_code(kernel)
    st, ws_bytes = decode_workspace_query(B, H, H_kv, Sq, d, bs, mb, nb, max_seq_len, mask, dt, kc)
    _check(st, "fa_decode_workspace_query")
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sp = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = decode_raw(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                    seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                    workspace.numel(), B, H, H_kv, Sq, d, bs, mb, nb, max_seq_len, float(scale),
                    mask_code(mask), dt, sp, kc)
    _check(st, "fa_decode_paged")
    return out, lse


def bwd_workspace_query(B, H, H_kv, Sq, Sk, d, mask="none", window=0, dtype=DTYPE_BF16):
    """(status, bytes) of fa_bwd_workspace_query."""
    n = ctypes.c_size_t(12345)
    st = load().fa_bwd_workspace_query(int(B), int(H), int(H_kv), int(Sq), int(Sk), int(d),
                                       mask_code(mask), int(window), int(dtype), ctypes.byref(n))
    return st, n.value


def workspace_query(B, H, Sq, Sk, d, mask="none", window=0, dtype=DTYPE_BF16):
    """(status, bytes) of fa_workspace_query."""
    n = ctypes.c_size_t(12345)
    st = load().fa_workspace_query(int(B), int(H), int(Sq), int(Sk), int(d), mask_code(mask),
                                   int(window), int(dtype), ctypes.byref(n))
    return st, n.value


def describe(d: int, mask="none", dtype=DTYPE_BF16) -> str:
    buf = ctypes.create_string_buffer(256)
    st = load().fa_describe(int(d), mask_code(mask), int(dtype), buf, 256)
    _check(st, "fa_describe")
    return buf.value.decode()


def device_error() -> int:
    return load().fa_get_device_error()


def set_debug_stall_ms(ms: int) -> None:
    """Test hook (fa_set_debug_stall_ms): with ms > 0 every later launch's
    first pipeline wait runs out after ms; 0 turns it off."""
    _check(load().fa_set_debug_stall_ms(int(ms)), "fa_set_debug_stall_ms")


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float16:
        return DTYPE_FP16
    raise FAError(FA_ERR_UNSUPPORTED, f"dtype {t.dtype} is not supported (bf16 / fp16 only)")


def forward(q, k, v, scale: float | None = None, mask="none", window: int = 0,
            out=None, lse=None, stream=None):
    """Fused attention forward on CUDA tensors [B, H, S, d] (bf16 or fp16).

    k and v may carry fewer heads than q (grouped-query attention: [B, H_kv,
    Sk, d] with H_kv dividing H, query head h reading K/V head h // (H //
    H_kv)); that case goes through fa_fwd_gqa, the rest through fa_fwd /
    fa_fwd_fp16.
    Returns (o, lse): o like q, lse fp32 [B, H, Sq].  Enqueued on ``stream``
    (default: torch's current stream of q's device); raises FAError if the
    library rejects the call.
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous [B,H,S,d] tensor")
    if not (q.dtype == k.dtype == v.dtype):
        raise FAError(FA_ERR_INVALID_ARG, "q, k, v must share one dtype")
    dt = _dtype_code(q)
    B, H, Sq, d = q.shape
    H_kv, Sk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, H_kv, Sk, d) or tuple(v.shape) != (B, H_kv, Sk, d):
        raise FAError(FA_ERR_INVALID_ARG, "k and v must be [B,H_kv,Sk,d] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sp = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if H_kv == H:
        st = fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                     B, H, Sq, Sk, d, float(scale), mask_code(mask), int(window), sp, dt)
        _check(st, "fa_fwd")
    else:
        st = fwd_gqa_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                         lse.data_ptr(), B, H, H_kv, Sq, Sk, d, float(scale), mask_code(mask),
                         int(window), sp, dt)
        _check(st, "fa_fwd_gqa")
    return out, lse


def backward(q, k, v, o, lse, dout, scale: float | None = None, mask="none", window: int = 0,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Attention backward on CUDA tensors (fa_bwd): returns (dq, dk, dv).

    q, o, dout [B, H, Sq, d]; k, v [B, H_kv, Sk, d] (bf16 or fp16, one dtype);
    lse fp32 [B, H, Sq] from ``forward`` with the same scale, mask and window.
    The workspace (a uint8 CUDA tensor) is allocated here unless given.
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("lse", lse)):
        if not t.is_cuda:
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be contiguous")
    if not (q.dtype == k.dtype == v.dtype == o.dtype == dout.dtype):
        raise FAError(FA_ERR_INVALID_ARG, "q, k, v, o, dout must share one dtype")
    if lse.dtype != torch.float32:
        raise FAError(FA_ERR_INVALID_ARG, "lse must be float32")
    dt = _dtype_code(q)
    B, H, Sq, d = q.shape
    H_kv, Sk = k.shape[1], k.shape[2]
    if (tuple(k.shape) != (B, H_kv, Sk, d) or tuple(v.shape) != (B, H_kv, Sk, d)
            or tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape)
            or tuple(lse.shape) != (B, H, Sq)):
        raise FAError(FA_ERR_INVALID_ARG, "shapes: q, o, dout [B,H,Sq,d]; k, v [B,H_kv,Sk,d]; lse [B,H,Sq]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st, ws_bytes = bwd_workspace_query(B, H, H_kv, Sq, Sk, d, mask, window, dt)
    _check(st, "fa_bwd_workspace_query")
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sp = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = bwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                 dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
                 workspace.numel(), B, H, H_kv, Sq, Sk, d, float(scale), mask_code(mask),
                 int(window), sp, dt)
    _check(st, "fa_bwd")
    return dq, dk, dv


def fwd_host_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, ws_ptr, ws_bytes, B, H, H_kv, Sq, Sk, d,
                 scale, mask_code_, window, dtype, stream_ptr) -> int:
    """fa_fwd_host with raw pointers (host buffers, device workspace)."""
    return load().fa_fwd_host(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, ws_ptr, ws_bytes, B, H, H_kv,
                              Sq, Sk, d, scale, mask_code_, window, dtype, stream_ptr)


def host_workspace_query(B, H, H_kv, Sq, Sk, d, mask="none", window=0, dtype=DTYPE_BF16):
    n = ctypes.c_size_t(0)
    st = load().fa_fwd_host_workspace_query(B, H, H_kv, Sq, Sk, d, mask_code(mask), int(window),
                                            dtype, ctypes.byref(n))
    return st, n.value


def forward_host(q, k, v, scale: float | None = None, mask="none", window: int = 0,
                 out=None, lse=None, workspace=None, device=None, stream=None, sync: bool = True):
    """End to end from host (CPU) tensors through fa_fwd_host: the library
    copies Q, K, V in, runs the forward and copies O and lse out, chunk by
    chunk with the copies overlapping the kernels.

    q [B, H, Sq, d], k and v [B, H_kv, Sk, d] CPU tensors (bf16 or fp16;
    pinned memory for asynchronous copies).  ``out`` / ``lse``: CPU tensors to
    write (allocated pinned here if not given); ``workspace``: a uint8 CUDA
    tensor of at least ``host_workspace_query`` bytes (allocated here if not
    given).  With sync=False the call returns once enqueued on ``stream``.
    Returns (out, lse).
    """
    import torch
    dev = torch.device(device or "cuda")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.is_cuda:
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a host tensor (use forward)")
        if t.dim() != 4 or not t.is_contiguous():
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous [B,H,S,d] tensor")
    if not (q.dtype == k.dtype == v.dtype):
        raise FAError(FA_ERR_INVALID_ARG, "q, k, v must share one dtype")
    dt = _dtype_code(q)
    B, H, Sq, d = q.shape
    H_kv, Sk = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, H_kv, Sk, d) or tuple(v.shape) != (B, H_kv, Sk, d):
        raise FAError(FA_ERR_INVALID_ARG, "k and v must be [B,H_kv,Sk,d] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, pin_memory=True)
    if out.is_cuda or lse.is_cuda or tuple(out.shape) != tuple(q.shape) or \
            tuple(lse.shape) != (B, H, Sq) or out.dtype != q.dtype or lse.dtype != torch.float32:
        raise FAError(FA_ERR_INVALID_ARG, "out / lse must be host tensors like q / [B,H,Sq] fp32")
    st, ws_bytes = host_workspace_query(B, H, H_kv, Sq, Sk, d, mask, window, dt)
    _check(st, "fa_fwd_host_workspace_query")
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    sp = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = fwd_host_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                      workspace.data_ptr(), workspace.numel(), B, H, H_kv, Sq, Sk, d, float(scale),
                      mask_code(mask), int(window), dt, sp)
    _check(st, "fa_fwd_host")
    if sync:
        stream.synchronize()
    return out, lse


# --------------------------------------------------- rotary positions and the 8-bit paged cache

def _enter(dev, stream):
    """Makes a call run on the tensors' own device and on ``stream``.

    Returns (raw stream pointer, scope to leave afterwards or None).  Outputs
    and workspaces made inside the scope are allocated for that stream, so the
    allocator cannot hand their memory to work of another stream too early.
    """
    import torch
    if stream is None:
        if torch._C._cuda_getDevice() == dev.index:
            return torch._C._cuda_getCurrentRawStream(dev.index), None
        scope = torch.cuda.device(dev)
        scope.__enter__()
        return torch._C._cuda_getCurrentRawStream(dev.index), scope
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else \
            torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise FAError(FA_ERR_INVALID_ARG, f"the stream is on {stream.device}, the tensors on {dev}")
    scope = torch.cuda.stream(stream)
    scope.__enter__()
    return stream.cuda_stream, scope


def _leave(scope):
    if scope is not None:
        scope.__exit__(None, None, None)


@functools.lru_cache(maxsize=256)
def _longs(values):
    """A host array of long long (never written to, so one per set of values will do)."""
    return (ctypes.c_longlong * len(values))(*values)


def _need_tensor(name, t, device, dtype, shape, contiguous=True):
    """Checks one tensor argument against what the call needs of it."""
    if t.device == device and t.dtype == dtype and t.shape == shape and (not contiguous or t.is_contiguous()):
        return
    if t.device != device:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be on {device}, it is on {t.device}")
    if t.dtype != dtype:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be {dtype}, it is {t.dtype}")
    if t.shape != shape:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must have shape {tuple(shape)}, it has {tuple(t.shape)}")
    raise FAError(FA_ERR_INVALID_ARG, f"{name} must be contiguous")


RopePlan = collections.namedtuple("RopePlan", "rot_dim freq amplitude")
RopePlan.__doc__ = """What ``rope`` needs of a model's rotary positions (made by ``rope_plan``):
the rotated components, their frequencies (device int64, turns per position
times 2^64) and the amplitude."""


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: float = 0.0, low_turns: float = 1.0, high_turns: float = 32.0):
    """(list of rot_dim / 2 integers: turns per position * 2^64, amplitude), by fa_rope_frequencies."""
    if scaling not in ROPE_SCALINGS:
        raise FAError(FA_ERR_UNSUPPORTED, f"scaling {scaling!r}: one of {list(ROPE_SCALINGS)}")
    freq = (ctypes.c_ulonglong * max(1, int(rot_dim) // 2))()
    amplitude = ctypes.c_float(0.0)
    st = load().fa_rope_frequencies(int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                    float(original_length), float(low_turns), float(high_turns), freq,
                                    ctypes.byref(amplitude))
    _check(st, "fa_rope_frequencies")
    return list(freq), amplitude.value


def rope_plan(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
              original_length: float = 0.0, low_turns: float = 1.0, high_turns: float = 32.0,
              device="cuda") -> RopePlan:
    """The frequencies of rotary positions over the first ``rot_dim`` components.

    scaling: "none"; "linear" (positions divided by ``factor``); "ntk" (the
    base grown so that the slowest pair is stretched by ``factor``);
    "by_parts" (pairs of at most ``low_turns`` turns over ``original_length``
    positions are stretched by ``factor``, those of at least ``high_turns``
    kept, and the amplitude is 0.1 ln(factor) + 1).
    """
    import torch
    freq, amplitude = rope_frequencies(rot_dim, base, scaling, factor, original_length, low_turns, high_turns)
    return RopePlan(int(rot_dim), torch.tensor(freq, dtype=torch.int64).to(device), amplitude)


_ROPE_DTYPES: dict = {}


def _rope_dtype(t) -> int:
    if not _ROPE_DTYPES:
        import torch
        _ROPE_DTYPES.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32})
    if t.dtype not in _ROPE_DTYPES:
        raise FAError(FA_ERR_UNSUPPORTED, f"dtype {t.dtype} is not supported (bf16 / fp16 / fp32 only)")
    return _ROPE_DTYPES[t.dtype]


def _rope(q, k, plan, positions, offset, layout, out_q, out_k, stream, direction):
    import torch
    lay = ROPE_LAYOUTS.get(layout)
    if lay is None:
        raise FAError(FA_ERR_UNSUPPORTED, f"layout {layout!r}: one of {list(ROPE_LAYOUTS)}")
    rot_dim, freq, amplitude = plan
    if freq.dtype != torch.int64 or not freq.is_contiguous() or 2 * freq.numel() < rot_dim:
        raise FAError(FA_ERR_INVALID_ARG, f"the plan's frequencies must be {rot_dim // 2} contiguous int64")
    dt = _rope_dtype(q)
    dev, dtype = q.device, q.dtype
    if not q.is_cuda or q.dim() != 4:
        raise FAError(FA_ERR_INVALID_ARG, "q must be a 4-D CUDA tensor [B,H,S,d]")
    B, H, S, d = q_shape = q.shape
    Hkv = 0
    if k is not None:
        k_shape = k.shape
        if len(k_shape) != 4 or k_shape[0] != B or k_shape[2] != S or k_shape[3] != d:
            raise FAError(FA_ERR_INVALID_ARG, "k must be [B,H_kv,S,d] matching q")
        Hkv = k_shape[1]
        _need_tensor("k", k, dev, dtype, k_shape, contiguous=False)
    elif out_k is not None:
        raise FAError(FA_ERR_INVALID_ARG, "out_k without k")
    if out_q is not None:
        _need_tensor("out_q", out_q, dev, dtype, q_shape, contiguous=False)
    if out_k is not None:
        _need_tensor("out_k", out_k, dev, dtype, k_shape, contiguous=False)
    if freq.device != dev:
        raise FAError(FA_ERR_INVALID_ARG, f"the plan is on {freq.device}, the tensors on {dev}")
    pos_ptr, pos_stride = None, 0
    if positions is not None:
        if positions.dtype != torch.int32 or positions.device != dev:
            raise FAError(FA_ERR_INVALID_ARG, f"positions must be int32 on {dev}")
        steps = positions.stride()
        if positions.shape == (B, S):
            pos_stride = steps[0] if B > 1 else 0
        elif positions.shape != (S,):
            raise FAError(FA_ERR_INVALID_ARG, "positions must be [B,S] or [S]")
        if S > 1 and steps[-1] != 1:
            raise FAError(FA_ERR_INVALID_ARG, "positions: the last dimension must be contiguous")
        pos_ptr = positions.data_ptr()
    sp, scope = _enter(dev, stream)
    try:
        if out_q is None:
            out_q = torch.empty(q_shape, dtype=dtype, device=dev)
        if k is not None and out_k is None:
            out_k = torch.empty(k_shape, dtype=dtype, device=dev)
        if B == 0 or S == 0 or d == 0 or H == 0:
            if k is None or k.numel() == 0:
                return out_q if k is None else (out_q, out_k)
            raise FAError(FA_ERR_INVALID_ARG, "q has no heads, k has some")
        q_steps, oq_steps, k_steps, ok_steps = q.stride(), out_q.stride(), None, None
        if Hkv:
            k_steps, ok_steps = k.stride(), out_k.stride()
        for steps in (q_steps, oq_steps, k_steps, ok_steps):
            if steps is not None and steps[3] != 1:
                raise FAError(FA_ERR_INVALID_ARG, "q, k and the outputs: the last dimension must be contiguous")
        st = (_lib or load()).fa_rope(
            q.data_ptr(), _longs(q_steps), out_q.data_ptr(), _longs(oq_steps),
            k.data_ptr() if Hkv else None, _longs(k_steps) if Hkv else None,
            out_k.data_ptr() if Hkv else None, _longs(ok_steps) if Hkv else None,
            pos_ptr, pos_stride, int(offset), freq.data_ptr(), amplitude, B, H, Hkv, S, d,
            rot_dim, lay, direction, dt, sp)
    finally:
        _leave(scope)
    if st:
        _check(st, "fa_rope")
    return out_q if k is None else (out_q, out_k)


def rope(q, k, plan: RopePlan, positions=None, offset: int = 0, layout: str = "half", out_q=None,
         out_k=None, stream=None):
    """Rotary positions on q [B, H, S, d] and k [B, H_kv, S, d] (k may be None), by fa_rope.

    Any strides with the last dimension contiguous (bf16, fp16 or fp32);
    ``positions`` int32 [B, S] or [S] (None: 0 .. S-1), ``offset`` added to
    them; ``layout`` "half" or "interleaved".  The outputs are contiguous
    unless given; ``out_q=q`` works in place.  Returns (q', k'), or q' alone
    without k.
    """
    return _rope(q, k, plan, positions, offset, layout, out_q, out_k, stream, ROPE_FORWARD)


def rope_backward(dq, dk, plan: RopePlan, positions=None, offset: int = 0, layout: str = "half",
                  out_q=None, out_k=None, stream=None):
    """Gradients of ``rope``'s inputs from those of its outputs; arguments as for ``rope``."""
    return _rope(dq, dk, plan, positions, offset, layout, out_q, out_k, stream, ROPE_BACKWARD)


PagedStep = collections.namedtuple("PagedStep", "seq_lens ring_state slot_map positions status")
PagedStep.__doc__ = """What ``paged_update`` returns: the new lengths [B] and ring state [2], the slot
and position of every row [max_tokens], and the status of every request [B]
(PAGED_OK, PAGED_NO_BLOCKS, PAGED_TOO_LONG or PAGED_NO_ROWS); int32."""


def paged_update(seq_lens, delta, block_table, free_ring, ring_state, block_size: int,
                 max_tokens: int | None = None, seq_lens_out=None, ring_state_out=None, slot_map=None,
                 positions=None, status=None, stream=None, rows_per_request: int | None = None) -> PagedStep:
    """One step of a paged cache's bookkeeping on the GPU (fa_paged_update, fa_paged_update_by_request).

    seq_lens and delta int32 [B] (tokens cached, and added or taken off);
    block_table int32 [B, max_blocks] and free_ring int32 [ring_size] are
    updated in place; ring_state int32 [2] is (head, count) of the free
    blocks.  ``max_tokens`` rows of slots and positions are written (given by
    slot_map's length if that is passed), the added tokens' one after the
    other.  With ``rows_per_request`` = n there are B * n rows instead, request
    b's tokens in the last of rows b * n .. b * n + n - 1 and slot -1 in the
    others: what a batch laid out by request, [B, heads, n, d], needs where a
    request may add fewer than n tokens, or none.  Outputs are allocated unless
    given; seq_lens_out and ring_state_out may be their inputs.
    """
    import torch
    if not seq_lens.is_cuda or seq_lens.dim() != 1 or block_table.dim() != 2 or free_ring.dim() != 1:
        raise FAError(FA_ERR_INVALID_ARG, "seq_lens [B] on a CUDA device, block_table [B,max_blocks], free_ring [n]")
    dev, i32 = seq_lens.device, torch.int32
    B, mb = seq_lens.shape[0], block_table.shape[1]
    call, rows = "fa_paged_update", max_tokens
    if rows_per_request is not None:
        call, rows = "fa_paged_update_by_request", int(rows_per_request)
        if max_tokens is not None and max_tokens != B * rows:
            raise FAError(FA_ERR_INVALID_ARG, f"max_tokens is {max_tokens}, B * rows_per_request {B * rows}")
        max_tokens = max(0, B * rows)
    if max_tokens is None:
        if slot_map is None and positions is None:
            raise FAError(FA_ERR_INVALID_ARG, "max_tokens, or slot_map, is needed")
        max_tokens = rows = (slot_map if slot_map is not None else positions).shape[0]
    _need_tensor("seq_lens", seq_lens, dev, i32, (B,))
    _need_tensor("delta", delta, dev, i32, (B,))
    _need_tensor("block_table", block_table, dev, i32, (B, mb))
    _need_tensor("free_ring", free_ring, dev, i32, free_ring.shape)
    _need_tensor("ring_state", ring_state, dev, i32, (2,))
    sp, scope = _enter(dev, stream)
    try:
        outs = []
        for name, t, n in (("seq_lens_out", seq_lens_out, B), ("ring_state_out", ring_state_out, 2),
                           ("slot_map", slot_map, max_tokens), ("positions", positions, max_tokens),
                           ("status", status, B)):
            if t is None:
                t = torch.empty(n, dtype=i32, device=dev)
            else:
                _need_tensor(name, t, dev, i32, (n,))
            outs.append(t)
        st = getattr(_lib or load(), call)(
            seq_lens.data_ptr(), delta.data_ptr(), block_table.data_ptr(), free_ring.data_ptr(),
            ring_state.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
            outs[3].data_ptr(), outs[4].data_ptr(), B, mb, free_ring.shape[0], int(block_size),
            int(rows), sp)
    finally:
        _leave(scope)
    _check(st, call)
    return PagedStep(*outs)


def _need_fp8_cache(k_cache, v_cache, k_scale, v_scale, dev):
    import torch
    dtype, shape = k_cache.dtype, k_cache.shape
    if len(shape) != 4 or dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise FAError(FA_ERR_INVALID_ARG,
                      "k_cache must be [num_blocks,H_kv,block_size,d], uint8 codes or float8_e4m3fn")
    heads = shape[:2]
    _need_tensor("k_cache", k_cache, dev, dtype, shape)
    _need_tensor("v_cache", v_cache, dev, dtype, shape)
    _need_tensor("k_scale", k_scale, dev, torch.float32, heads)
    _need_tensor("v_scale", v_scale, dev, torch.float32, heads)


def cache_append_fp8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """Quantises new K and V rows into an 8-bit paged cache, in place (fa_cache_append_fp8).

    k, v [T, H_kv, d] (bf16 or fp16; any strides with the last dimension
    contiguous); slot_map int32 [T] (negative: the row is skipped; the rows of
    one block stand together); k_cache, v_cache [num_blocks, H_kv, block_size,
    d] of e4m3 (uint8 codes or float8_e4m3fn); k_scale, v_scale fp32
    [num_blocks, H_kv].
    """
    import torch
    if not k.is_cuda or k.dim() != 3 or k_cache.dim() != 4:
        raise FAError(FA_ERR_INVALID_ARG, "k must be a CUDA tensor [T,H_kv,d], the caches [blocks,H_kv,bs,d]")
    dev = k.device
    dt = _dtype_code(k)
    T, Hkv, d = k.shape
    nb, hc, bs, dc = k_cache.shape
    _need_tensor("v", v, dev, k.dtype, k.shape, contiguous=False)
    if (hc, dc) != (Hkv, d):
        raise FAError(FA_ERR_INVALID_ARG, "the caches' heads and components must be those of k")
    if k.numel() and (k.stride(2) != 1 or v.stride(2) != 1):
        raise FAError(FA_ERR_INVALID_ARG, "k and v: the last dimension must be contiguous")
    _need_tensor("slot_map", slot_map, dev, torch.int32, (T,))
    _need_fp8_cache(k_cache, v_cache, k_scale, v_scale, dev)
    sp, scope = _enter(dev, stream)
    try:
        st = (_lib or load()).fa_cache_append_fp8(
            k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
            slot_map.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), T, Hkv, d, bs, nb, dt, sp)
    finally:
        _leave(scope)
    _check(st, "fa_cache_append_fp8")


def decode_fp8_workspace_query(B, H, H_kv, Sq, d, block_size, max_blocks, num_blocks, max_seq_len,
                               mask="none", dtype=DTYPE_BF16):
    """(status, bytes) of fa_decode_fp8_workspace_query."""
    n = ctypes.c_size_t(12345)
    st = load().fa_decode_fp8_workspace_query(int(B), int(H), int(H_kv), int(Sq), int(d), int(block_size),
                                              int(max_blocks), int(num_blocks), int(max_seq_len),
                                              mask_code(mask), int(dtype), ctypes.byref(n))
    return st, n.value


@functools.lru_cache(maxsize=1024)
def _decode_fp8_workspace(device_index, *sizes):
    """Workspace bytes for these sizes on this device (the current one); refusals are not kept."""
    n = ctypes.c_size_t(0)
    _check(load().fa_decode_fp8_workspace_query(*sizes, ctypes.byref(n)), "fa_decode_fp8_workspace_query")
    return n.value


def decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_seq_len: int,
                     scale: float | None = None, mask="none", out=None, lse=None, workspace=None,
                     stream=None):
    """Attention of q's new rows over an 8-bit paged cache (fa_decode_paged_fp8).

    q [B, H, Sq, d] bf16 or fp16; the caches and scales as ``cache_append_fp8``
    writes them; block_table int32 [B, max_blocks], seq_lens int32 [B] (0
    allowed: the row's output is 0 and its lse -inf).  Returns (o, lse).
    """
    import torch
    q_shape, c_shape, t_shape = q.shape, k_cache.shape, block_table.shape
    if not q.is_cuda or len(q_shape) != 4 or not q.is_contiguous() or len(c_shape) != 4:
        raise FAError(FA_ERR_INVALID_ARG, "q must be a contiguous CUDA tensor [B,H,Sq,d], the caches 4-D")
    dev = q.device
    dt = _dtype_code(q)
    B, H, Sq, d = q_shape
    nb, Hkv, bs, dc = c_shape
    if dc != d or len(t_shape) != 2:
        raise FAError(FA_ERR_INVALID_ARG, "the caches' last dimension must be q's; block_table [B,max_blocks]")
    mb = t_shape[1]
    _need_tensor("block_table", block_table, dev, torch.int32, (B, mb))
    _need_tensor("seq_lens", seq_lens, dev, torch.int32, (B,))
    _need_fp8_cache(k_cache, v_cache, k_scale, v_scale, dev)
    mk = mask_code(mask)
    if scale is None:
        scale = d ** -0.5
    max_seq_len = int(max_seq_len)
    sp, scope = _enter(dev, stream)
    try:
        if workspace is None:
            ws_bytes = _decode_fp8_workspace(dev.index, B, H, Hkv, Sq, d, bs, mb, nb, max_seq_len, mk, dt)
            if ws_bytes:
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        else:
            _need_tensor("workspace", workspace, dev, torch.uint8, workspace.shape)
            ws_bytes = workspace.numel()
        if out is None:
            out = torch.empty_like(q)
        else:
            _need_tensor("out", out, dev, q.dtype, q_shape)
        if lse is None:
            lse = torch.empty((B, H, Sq), dtype=torch.float32, device=dev)
        else:
            _need_tensor("lse", lse, dev, torch.float32, (B, H, Sq))
        st = (_lib or load()).fa_decode_paged_fp8(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(),
            workspace.data_ptr() if ws_bytes else None, ws_bytes, B, H, Hkv, Sq, d, bs, mb, nb,
            max_seq_len, scale, mk, dt, sp)
    finally:
        _leave(scope)
    if st:
        _check(st, "fa_decode_paged_fp8")
    return out, lse


# --------------------------------------------------------------- the paged cache in 4 bits

def int4_cache(num_blocks: int, H_kv: int, block_size: int, d: int, group: int = 32, device="cuda"):
    """An empty 4-bit paged cache: (k_cache, v_cache, k_scale, v_scale), all zeros.

    The caches are uint8 [num_blocks, H_kv, block_size, d / 2], two codes to a
    byte; the scales int32 words [num_blocks, H_kv, block_size, d / group], a
    group's scale (bf16) in the high half and its zero (fp16) in the low one.
    """
    import torch
    if d not in (64, 128, 256) or group not in (32, 64) or block_size not in (16, 32, 64, 128):
        raise FAError(FA_ERR_UNSUPPORTED, "d must be 64, 128 or 256, group 32 or 64, block_size 16, 32, 64 or 128")
    rows = (int(num_blocks), int(H_kv), int(block_size))
    return (*(torch.zeros((*rows, d // 2), dtype=torch.uint8, device=device) for _ in range(2)),
            *(torch.zeros((*rows, d // group), dtype=torch.int32, device=device) for _ in range(2)))


def _need_int4_cache(k_cache, v_cache, k_scale, v_scale, dev):
    """Checks the four tensors of a 4-bit cache; returns (num_blocks, H_kv, block_size, d, group)."""
    import torch
    shape, words = k_cache.shape, k_scale.shape
    if len(shape) != 4 or len(words) != 4:
        raise FAError(FA_ERR_INVALID_ARG, "the caches must be [num_blocks,H_kv,block_size,d/2], the scales "
                                          "[num_blocks,H_kv,block_size,d/group]")
    d = 2 * shape[3]
    if words[3] < 1 or d % words[3]:
        raise FAError(FA_ERR_INVALID_ARG, f"{words[3]} scales per row do not divide {d} components into groups")
    want = (*shape[:3], words[3])
    _need_tensor("k_cache", k_cache, dev, torch.uint8, shape)
    _need_tensor("v_cache", v_cache, dev, torch.uint8, shape)
    _need_tensor("k_scale", k_scale, dev, torch.int32, want)
    _need_tensor("v_scale", v_scale, dev, torch.int32, want)
    return shape[0], shape[1], shape[2], d, d // words[3]


def cache_append_int4(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """Quantises new K and V rows into a 4-bit paged cache, in place (fa_cache_append_int4).

    k, v [T, H_kv, d] (bf16 or fp16; any strides with the last dimension
    contiguous); slot_map int32 [T] (negative: the row is skipped); the caches
    and scales as ``int4_cache`` makes them.
    """
    import torch
    if not k.is_cuda or k.dim() != 3:
        raise FAError(FA_ERR_INVALID_ARG, "k must be a CUDA tensor [T,H_kv,d]")
    dev = k.device
    dt = _dtype_code(k)
    T, Hkv, d = k.shape
    _need_tensor("v", v, dev, k.dtype, k.shape, contiguous=False)
    nb, hc, bs, dc, group = _need_int4_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if (hc, dc) != (Hkv, d):
        raise FAError(FA_ERR_INVALID_ARG, "the caches' heads and components must be those of k")
    if k.numel() and (k.stride(2) != 1 or v.stride(2) != 1):
        raise FAError(FA_ERR_INVALID_ARG, "k and v: the last dimension must be contiguous")
    _need_tensor("slot_map", slot_map, dev, torch.int32, (T,))
    sp, scope = _enter(dev, stream)
    try:
        st = (_lib or load()).fa_cache_append_int4(
            k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
            slot_map.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), T, Hkv, d, group, bs, nb, dt, sp)
    finally:
        _leave(scope)
    _check(st, "fa_cache_append_int4")


def cache_read_int4(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, rows: int, starts=None,
                    dtype=None, out_k=None, out_v=None, stream=None):
    """Reads rows of a 4-bit paged cache back in 16 bits (fa_cache_read_int4).

    Row i of request b is its token ``starts[b] + i`` (starts int32 [B]; None: 0),
    i < rows.  Returns (k, v) [B, H_kv, rows, d], as ``forward`` takes them.
    Rows without a token are zeros, or stay as they were in ``out_k`` and
    ``out_v`` (bf16 or fp16; any strides with the last dimension contiguous;
    both or none).  ``dtype`` is the outputs' where they are not given (bf16).
    """
    import torch
    if not k_cache.is_cuda or block_table.dim() != 2:
        raise FAError(FA_ERR_INVALID_ARG, "the caches must be CUDA tensors, block_table [B,max_blocks]")
    dev = k_cache.device
    nb, Hkv, bs, d, group = _need_int4_cache(k_cache, v_cache, k_scale, v_scale, dev)
    B, mb = block_table.shape
    rows = int(rows)
    if rows < 0 or (out_k is None) != (out_v is None):
        raise FAError(FA_ERR_INVALID_ARG, "rows must be >= 0, and out_k and out_v given both or not at all")
    _need_tensor("block_table", block_table, dev, torch.int32, (B, mb))
    _need_tensor("seq_lens", seq_lens, dev, torch.int32, (B,))
    if starts is not None:
        _need_tensor("starts", starts, dev, torch.int32, (B,))
    shape = (B, Hkv, rows, d)
    sp, scope = _enter(dev, stream)
    try:
        if out_k is None:
            dtype = dtype or torch.bfloat16
            out_k, out_v = (torch.zeros(shape, dtype=dtype, device=dev) for _ in range(2))
        dt = _dtype_code(out_k)
        if dtype is not None and out_k.dtype != dtype:
            raise FAError(FA_ERR_INVALID_ARG, f"out_k is {out_k.dtype}, dtype {dtype}")
        _need_tensor("out_k", out_k, dev, out_k.dtype, shape, contiguous=False)
        _need_tensor("out_v", out_v, dev, out_k.dtype, shape, contiguous=False)
        if rows and B and (out_k.stride(3) != 1 or out_v.stride(3) != 1):
            raise FAError(FA_ERR_INVALID_ARG, "out_k and out_v: the last dimension must be contiguous")
        st = (_lib or load()).fa_cache_read_int4(
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), None if starts is None else starts.data_ptr(),
            out_k.data_ptr(), _longs(out_k.stride()[:3]), out_v.data_ptr(), _longs(out_v.stride()[:3]),
            B, Hkv, rows, d, group, bs, mb, nb, dt, sp)
    finally:
        _leave(scope)
    _check(st, "fa_cache_read_int4")
    return out_k, out_v


def decode_int4_workspace_query(B, H, H_kv, Sq, d, group, block_size, max_blocks, num_blocks, max_seq_len,
                                mask="none", dtype=DTYPE_BF16):
    """(status, bytes) of fa_decode_int4_workspace_query."""
    n = ctypes.c_size_t(12345)
    st = load().fa_decode_int4_workspace_query(int(B), int(H), int(H_kv), int(Sq), int(d), int(group),
                                               int(block_size), int(max_blocks), int(num_blocks),
                                               int(max_seq_len), mask_code(mask), int(dtype), ctypes.byref(n))
    return st, n.value


@functools.lru_cache(maxsize=1024)
def _decode_int4_workspace(device_index, *sizes):
    """Workspace bytes for these sizes on this device (the current one); refusals are not kept."""
    n = ctypes.c_size_t(0)
    _check(load().fa_decode_int4_workspace_query(*sizes, ctypes.byref(n)), "fa_decode_int4_workspace_query")
    return n.value


def decode_paged_int4(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, max_seq_len: int,
                      scale: float | None = None, mask="none", out=None, lse=None, workspace=None,
                      stream=None):
    """Attention of q's new rows over a 4-bit paged cache (fa_decode_paged_int4).

    q [B, H, Sq, d] bf16 or fp16; the caches and scales as ``cache_append_int4``
    writes them; block_table int32 [B, max_blocks], seq_lens int32 [B] (0
    allowed: the row's output is 0 and its lse -inf).  Returns (o, lse).
    """
    import torch
    q_shape, t_shape = q.shape, block_table.shape
    if not q.is_cuda or len(q_shape) != 4 or not q.is_contiguous() or len(t_shape) != 2:
        raise FAError(FA_ERR_INVALID_ARG, "q must be a contiguous CUDA tensor [B,H,Sq,d], block_table [B,max_blocks]")
    dev = q.device
    dt = _dtype_code(q)
    B, H, Sq, d = q_shape
    nb, Hkv, bs, dc, group = _need_int4_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if dc != d:
        raise FAError(FA_ERR_INVALID_ARG, f"the caches hold rows of {dc} components, q of {d}")
    mb = t_shape[1]
    _need_tensor("block_table", block_table, dev, torch.int32, (B, mb))
    _need_tensor("seq_lens", seq_lens, dev, torch.int32, (B,))
    mk = mask_code(mask)
    if scale is None:
        scale = d ** -0.5
    max_seq_len = int(max_seq_len)
    sp, scope = _enter(dev, stream)
    try:
        if workspace is None:
            ws_bytes = _decode_int4_workspace(dev.index, B, H, Hkv, Sq, d, group, bs, mb, nb, max_seq_len, mk, dt)
            if ws_bytes:
                workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        else:
            _need_tensor("workspace", workspace, dev, torch.uint8, workspace.shape)
            ws_bytes = workspace.numel()
        if out is None:
            out = torch.empty_like(q)
        else:
            _need_tensor("out", out, dev, q.dtype, q_shape)
        if lse is None:
            lse = torch.empty((B, H, Sq), dtype=torch.float32, device=dev)
        else:
            _need_tensor("lse", lse, dev, torch.float32, (B, H, Sq))
        st = (_lib or load()).fa_decode_paged_int4(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(),
            workspace.data_ptr() if ws_bytes else None, ws_bytes, B, H, Hkv, Sq, d, group, bs, mb, nb,
            max_seq_len, scale, mk, dt, sp)
    finally:
        _leave(scope)
    if st:
        _check(st, "fa_decode_paged_int4")
    return out, lse
