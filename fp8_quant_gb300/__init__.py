"""GB300 KV-cache write path: Python binding of ``libkvstore.so``.

The library (the kernels in ``csrc/*.cu``, C ABI in ``include/kvstore.h``) does
all the work; this module only marshals arguments. It exposes the C entry points under
the same names:

* :func:`kv_store`      -- plain byte-exact scatter of K/V rows into cache slots
  (sglang ``kvcache.cuh``, ``store_kvcache``).
* :func:`kv_store_fp8`  -- fused fp32 scale + FP8 e4m3fn conversion + paged
  scatter (sglang ``trtllm_fp8_kv_kernel.py``, ``fused_fp8_set_kv_buffer``).
* :func:`kv_store_paged`, :func:`kv_store_fp8_ex` (e5m2; scales per tensor, or
  per token row / per (token, head) computed in the kernel),
  :func:`kv_gather`, :func:`kv_gather_fp8` (the inverse), :func:`kv_inv_scale`,
  :func:`kv_absmax_inv` (scale preparation), :func:`kv_store_fp8_dynamic_tensor`
  (per-tensor scales formed from the batch and the write, in one call).
* :func:`kv_store_rope` (append with the position rotation applied on the way;
  16-bit, e4m3fn or 4-bit e2m1 caches), :func:`kv_gather_fp4` (the 4-bit
  cache's read-back), :func:`kv_attend` (attention over those caches).
* :func:`kv_store_latent`, :func:`kv_gather_latent`, :func:`kv_attend_latent` (a cache
  of latent rows, which all query heads share as keys and values: its append, its
  read-back and attention over it; 16-bit or e4m3fn rows).
* :func:`kv_error_poll`, :func:`kv_error_reset`, :func:`kv_status_str`.

The tensor-level functions take torch tensors (device memory and streams come
from PyTorch) and pass their data pointers and byte strides; the ``raw``
functions take plain integers exactly as the C ABI does. There is no CPU
fallback: if the compiled library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import enum
import math
import os
import threading
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libkvstore.so")

__all__ = [
    "KVStatus", "KVError", "kv_store", "kv_store_fp8", "kv_store_paged", "kv_store_fp8_ex",
    "kv_gather", "kv_gather_fp8", "kv_inv_scale", "kv_absmax_inv", "kv_error_poll",
    "kv_error_reset", "kv_status_str", "error_record", "load_library", "raw", "STRIDE_FIELDS",
    "fused_fp8_set_kv_buffer", "kv_store_fp8_dynamic_tensor", "DYNAMIC_TENSOR_WORK_BYTES",
    "kv_store_rope", "kv_gather_fp4", "kv_attend", "ATTEND_WORK_BYTES",
    "kv_store_latent", "kv_gather_latent", "kv_attend_latent",
]


class KVStatus(enum.IntEnum):
    OK = 0
    ERR_INVALID_ARG = 1
    ERR_UNSUPPORTED = 2
    ERR_CUDA = 3
    ERR_INDEX_OOB = 4
    ERR_WAIT = 5


class KVError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = KVStatus(status)
        super().__init__(f"{what}: {kv_status_str(status)}")


STRIDE_FIELDS = ("k_token", "k_head", "k_dim", "v_token", "v_head", "v_dim",
                 "kc_slot", "kc_head", "kc_dim", "vc_slot", "vc_head", "vc_dim")


class _Strides(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in STRIDE_FIELDS]


class _Rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("cos_sin_stride", ctypes.c_int64),
                ("max_position", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("position_dtype", ctypes.c_int32), ("position_stride", ctypes.c_int64),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("num_q_heads", ctypes.c_int32), ("q_token", ctypes.c_int64),
                ("q_head", ctypes.c_int64), ("qo_token", ctypes.c_int64),
                ("qo_head", ctypes.c_int64)]


class _BlockScales(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (f, ctypes.c_int64) for f in ("k_page", "k_slot", "k_head", "v_page", "v_slot", "v_head")]


class _AttendStrides(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in (
        "q_token", "q_head", "o_token", "o_head", "kc_page", "kc_slot", "kc_head",
        "vc_page", "vc_slot", "vc_head")]


class _LatentStrides(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in (
        "c_token", "r_token", "cache_page", "cache_slot", "scale_slot")]


class _AttendLatentStrides(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in (
        "q_token", "q_head", "o_token", "o_head", "cache_page", "cache_slot", "scale_slot")]


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load ``libkvstore.so`` (built by ``fp8_quant_gb300.build``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library {p} is missing: build it with `python -m fp8_quant_gb300.build` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        lib.kv_store.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                 ctypes.POINTER(_Strides), I64, I32, P, P]
        lib.kv_store.restype = I32
        lib.kv_store_fp8.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                     ctypes.POINTER(_Strides), I64, I64, I64, I64, P, P, I32, P, P]
        lib.kv_store_fp8.restype = I32
        lib.kv_store_paged.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                       ctypes.POINTER(_Strides), I64, I64, I64, I64, I32, P, P]
        lib.kv_store_paged.restype = I32
        lib.kv_gather.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                  ctypes.POINTER(_Strides), I64, P, P]
        lib.kv_gather.restype = I32
        lib.kv_gather_paged.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                        ctypes.POINTER(_Strides), I64, I64, I64, I64, P, P]
        lib.kv_gather_paged.restype = I32
        lib.kv_gather_fp8.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                      ctypes.POINTER(_Strides), I64, I64, I64, I64, P, P, I32, P,
                                      P]
        lib.kv_gather_fp8.restype = I32
        lib.kv_store_fp8_ex.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                        ctypes.POINTER(_Strides), I64, I64, I64, I64, I32, I32,
                                        P, P, P, P, I64, P, P]
        lib.kv_store_fp8_ex.restype = I32
        lib.kv_gather_fp8_ex.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                         ctypes.POINTER(_Strides), I64, I64, I64, I64, I32, I32,
                                         P, P, P, P, I64, P, P]
        lib.kv_gather_fp8_ex.restype = I32
        lib.kv_inv_scale.argtypes = [P, P, I64, P]
        lib.kv_inv_scale.restype = I32
        lib.kv_absmax_inv.argtypes = [P, P, I32, I64, I32, I32, ctypes.POINTER(_Strides),
                                      ctypes.c_float, P, P, P, P]
        lib.kv_absmax_inv.restype = I32
        lib.kv_store_fp8_dynamic_tensor.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                                    ctypes.POINTER(_Strides), I64, I64, I64, I64,
                                                    I32, P, P, P, P, P]
        lib.kv_store_fp8_dynamic_tensor.restype = I32
        lib.kv_store_rope.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                      ctypes.POINTER(_Strides), I64, I64, I64, I64,
                                      ctypes.POINTER(_Rope), I32, P, P,
                                      ctypes.POINTER(_BlockScales), P, P]
        lib.kv_store_rope.restype = I32
        lib.kv_gather_fp4.argtypes = [P, P, ctypes.POINTER(_BlockScales), P, P, P, I32, I64, I64,
                                      I32, I32, I32, ctypes.POINTER(_Strides), I64, I64, I64, I64,
                                      P, P, P, P]
        lib.kv_gather_fp4.restype = I32
        lib.kv_attend.argtypes = [P, P, P, P, P, P, I64, I64, P, P, I32, I64, I32, I32, I32, I32,
                                  ctypes.POINTER(_AttendStrides), I64, I64, I32, P, P,
                                  ctypes.POINTER(_BlockScales), ctypes.c_float, I64, I64, P, I64,
                                  P, P]
        lib.kv_attend.restype = I32
        lib.kv_store_latent.argtypes = [P, P, P, P, I32, I64, I64, I32, I32, I32,
                                        ctypes.POINTER(_LatentStrides), I64, I64, P, ctypes.c_float,
                                        ctypes.POINTER(_Rope), I32, P, P, P]
        lib.kv_store_latent.restype = I32
        lib.kv_gather_latent.argtypes = [P, P, P, P, I32, I64, I64, I32, I32,
                                         ctypes.POINTER(_LatentStrides), I64, I64, I32, P, P]
        lib.kv_gather_latent.restype = I32
        lib.kv_attend_latent.argtypes = [P, P, P, P, P, P, I64, I64, P, P, I32, I64, I32, I32, I32,
                                         I32, ctypes.POINTER(_AttendLatentStrides), I64, I64, I32,
                                         ctypes.c_float, P, I64, P, P]
        lib.kv_attend_latent.restype = I32
        lib.kv_store_noalloc.argtypes = [P, P, P, P, P, I32, I64, I64, I32, I32, I32,
                                         ctypes.POINTER(_Strides), I64, I32,
                                         ctypes.POINTER(I64), ctypes.POINTER(I64), P]
        lib.kv_store_noalloc.restype = I32
        lib.kv_error_poll.argtypes = [P, P, ctypes.POINTER(I64), ctypes.POINTER(I64)]
        lib.kv_error_poll.restype = I32
        lib.kv_error_snapshot.argtypes = [P, P, P]
        lib.kv_error_snapshot.restype = I32
        lib.kv_launch_floor.argtypes = [I64, P]
        lib.kv_launch_floor.restype = I32
        lib.kv_error_reset.argtypes = [P, P]
        lib.kv_error_reset.restype = I32
        lib.kv_status_str.argtypes = [I32]
        lib.kv_status_str.restype = ctypes.c_char_p
        lib.kv_last_cuda_error.argtypes = []
        lib.kv_last_cuda_error.restype = ctypes.c_int
        lib.kv_abi_version.argtypes = []
        lib.kv_abi_version.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def kv_status_str(status: int) -> str:
    return load_library().kv_status_str(int(status)).decode()


# ---------------------------------------------------------------------------
# Raw entry points: integers in, status out (the C ABI one to one).
# ---------------------------------------------------------------------------

class raw:
    """The C ABI with plain integers (device addresses, byte strides, stream handle)."""

    @staticmethod
    def kv_store(k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens,
                 num_heads, head_dim, elem_bytes, strides: Sequence[int], size_limit,
                 num_split, d_err, stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_store(k, v, k_cache, v_cache, indices, index_dtype,
                                       index_stride, num_tokens, num_heads, head_dim,
                                       elem_bytes, ctypes.byref(st), size_limit, num_split,
                                       d_err, stream)

    @staticmethod
    def kv_store_fp8(k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens,
                     num_heads, head_dim, src_dtype, strides: Sequence[int], page_size,
                     kc_page_stride, vc_page_stride, size_limit, inv_k_scale, inv_v_scale,
                     use_scale, d_err, stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_store_fp8(k, v, k_cache, v_cache, indices, index_dtype,
                                           index_stride, num_tokens, num_heads, head_dim,
                                           src_dtype, ctypes.byref(st), page_size,
                                           kc_page_stride, vc_page_stride, size_limit,
                                           inv_k_scale, inv_v_scale, use_scale, d_err, stream)

    @staticmethod
    def kv_store_paged(k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens,
                       num_heads, head_dim, elem_bytes, strides: Sequence[int], page_size,
                       kc_page_stride, vc_page_stride, size_limit, num_split, d_err,
                       stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_store_paged(k, v, k_cache, v_cache, indices, index_dtype,
                                             index_stride, num_tokens, num_heads, head_dim,
                                             elem_bytes, ctypes.byref(st), page_size,
                                             kc_page_stride, vc_page_stride, size_limit,
                                             num_split, d_err, stream)

    @staticmethod
    def kv_gather(k_cache, v_cache, k_out, v_out, indices, index_dtype, index_stride, num_tokens,
                  num_heads, head_dim, elem_bytes, strides: Sequence[int], size_limit, d_err,
                  stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_gather(k_cache, v_cache, k_out, v_out, indices, index_dtype,
                                        index_stride, num_tokens, num_heads, head_dim, elem_bytes,
                                        ctypes.byref(st), size_limit, d_err, stream)

    @staticmethod
    def kv_gather_paged(k_cache, v_cache, k_out, v_out, indices, index_dtype, index_stride,
                        num_tokens, num_heads, head_dim, elem_bytes, strides: Sequence[int],
                        page_size, kc_page_stride, vc_page_stride, size_limit, d_err,
                        stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_gather_paged(k_cache, v_cache, k_out, v_out, indices,
                                              index_dtype, index_stride, num_tokens, num_heads,
                                              head_dim, elem_bytes, ctypes.byref(st), page_size,
                                              kc_page_stride, vc_page_stride, size_limit, d_err,
                                              stream)

    @staticmethod
    def kv_gather_fp8(k_cache, v_cache, k_out, v_out, indices, index_dtype, index_stride,
                      num_tokens, num_heads, head_dim, out_dtype, strides: Sequence[int],
                      page_size, kc_page_stride, vc_page_stride, size_limit, k_scale, v_scale,
                      use_scale, d_err, stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_gather_fp8(k_cache, v_cache, k_out, v_out, indices, index_dtype,
                                            index_stride, num_tokens, num_heads, head_dim,
                                            out_dtype, ctypes.byref(st), page_size,
                                            kc_page_stride, vc_page_stride, size_limit, k_scale,
                                            v_scale, use_scale, d_err, stream)

    @staticmethod
    def kv_store_fp8_ex(k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens,
                        num_heads, head_dim, src_dtype, strides: Sequence[int], page_size,
                        kc_page_stride, vc_page_stride, size_limit, fmt, scale_mode, inv_k_scale,
                        inv_v_scale, k_scales, v_scales, scales_slot_stride, d_err,
                        stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_store_fp8_ex(k, v, k_cache, v_cache, indices, index_dtype,
                                              index_stride, num_tokens, num_heads, head_dim,
                                              src_dtype, ctypes.byref(st), page_size,
                                              kc_page_stride, vc_page_stride, size_limit, fmt,
                                              scale_mode, inv_k_scale, inv_v_scale, k_scales,
                                              v_scales, scales_slot_stride, d_err, stream)

    @staticmethod
    def kv_store_fp8_dynamic_tensor(k, v, k_cache, v_cache, indices, index_dtype, index_stride,
                                    num_tokens, num_heads, head_dim, src_dtype,
                                    strides: Sequence[int], page_size, kc_page_stride,
                                    vc_page_stride, size_limit, fmt, k_scale, v_scale, work,
                                    d_err, stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_store_fp8_dynamic_tensor(
            k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens, num_heads,
            head_dim, src_dtype, ctypes.byref(st), page_size, kc_page_stride, vc_page_stride,
            size_limit, fmt, k_scale, v_scale, work, d_err, stream)

    @staticmethod
    def kv_gather_fp8_ex(k_cache, v_cache, k_out, v_out, indices, index_dtype, index_stride,
                         num_tokens, num_heads, head_dim, out_dtype, strides: Sequence[int],
                         page_size, kc_page_stride, vc_page_stride, size_limit, fmt, scale_mode,
                         k_scale, v_scale, k_scales, v_scales, scales_slot_stride, d_err,
                         stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_gather_fp8_ex(k_cache, v_cache, k_out, v_out, indices,
                                               index_dtype, index_stride, num_tokens, num_heads,
                                               head_dim, out_dtype, ctypes.byref(st), page_size,
                                               kc_page_stride, vc_page_stride, size_limit, fmt,
                                               scale_mode, k_scale, v_scale, k_scales, v_scales,
                                               scales_slot_stride, d_err, stream)

    @staticmethod
    def kv_inv_scale(scale, inv, n, stream) -> int:
        return load_library().kv_inv_scale(scale, inv, n, stream)

    @staticmethod
    def kv_absmax_inv(k, v, src_dtype, num_tokens, num_heads, head_dim, strides: Sequence[int],
                      fp8_max, amax, inv, work, stream) -> int:
        st = _Strides(*[int(x) for x in strides])
        return load_library().kv_absmax_inv(k, v, src_dtype, num_tokens, num_heads, head_dim,
                                            ctypes.byref(st), float(fp8_max), amax, inv, work,
                                            stream)

    @staticmethod
    def kv_store_rope(k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens,
                      num_heads, head_dim, src_dtype, strides: Sequence[int], page_size,
                      kc_page_stride, vc_page_stride, size_limit, rope: Sequence, fmt,
                      inv_k_scale, inv_v_scale, scales: Optional[Sequence], d_err, stream) -> int:
        """``rope`` and ``scales``: the fields of kv_rope / kv_block_scales in order."""
        return load_library().kv_store_rope(
            k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_tokens, num_heads,
            head_dim, src_dtype, ctypes.byref(_Strides(*strides)), page_size, kc_page_stride,
            vc_page_stride, size_limit, None if rope is None else ctypes.byref(_Rope(*rope)), fmt,
            inv_k_scale, inv_v_scale,
            None if scales is None else ctypes.byref(_BlockScales(*scales)), d_err, stream)

    @staticmethod
    def kv_gather_fp4(k_cache, v_cache, scales: Optional[Sequence], k_out, v_out, indices,
                      index_dtype, index_stride, num_tokens, num_heads, head_dim, out_dtype,
                      strides: Sequence[int], page_size, kc_page_stride, vc_page_stride,
                      size_limit, k_scale, v_scale, d_err, stream) -> int:
        return load_library().kv_gather_fp4(
            k_cache, v_cache, None if scales is None else ctypes.byref(_BlockScales(*scales)),
            k_out, v_out, indices, index_dtype, index_stride, num_tokens, num_heads, head_dim,
            out_dtype, ctypes.byref(_Strides(*strides)), page_size, kc_page_stride,
            vc_page_stride, size_limit, k_scale, v_scale, d_err, stream)

    @staticmethod
    def kv_attend(q, out, lse, k_cache, v_cache, page_table, table_stride, table_width, seq_lens,
                  q_start, num_seqs, num_q_tokens, num_q_heads, num_heads, head_dim, dtype,
                  strides: Optional[Sequence[int]], page_size, num_pages, fmt, k_scale, v_scale,
                  scales: Optional[Sequence], sm_scale, window, sinks, work, work_bytes, d_err,
                  stream) -> int:
        return load_library().kv_attend(
            q, out, lse, k_cache, v_cache, page_table, table_stride, table_width, seq_lens,
            q_start, num_seqs, num_q_tokens, num_q_heads, num_heads, head_dim, dtype,
            None if strides is None else ctypes.byref(_AttendStrides(*strides)), page_size,
            num_pages, fmt, k_scale, v_scale,
            None if scales is None else ctypes.byref(_BlockScales(*scales)), sm_scale, window,
            sinks, work, work_bytes, d_err, stream)

    @staticmethod
    def kv_store_latent(c, r, cache, indices, index_dtype, index_stride, num_tokens, latent_dim,
                        rope_dim, src_dtype, strides: Optional[Sequence[int]], page_size,
                        size_limit, weight, eps, rope: Optional[Sequence], fmt, scales, d_err,
                        stream) -> int:
        """``strides`` and ``rope``: the fields of kv_latent_strides / kv_rope in order."""
        return load_library().kv_store_latent(
            c, r, cache, indices, index_dtype, index_stride, num_tokens, latent_dim, rope_dim,
            src_dtype, None if strides is None else ctypes.byref(_LatentStrides(*strides)), page_size,
            size_limit, weight, eps, None if rope is None else ctypes.byref(_Rope(*rope)), fmt, scales,
            d_err, stream)

    @staticmethod
    def kv_gather_latent(cache, scales, out, indices, index_dtype, index_stride, num_tokens,
                         row_dim, out_dtype, strides: Optional[Sequence[int]], page_size,
                         size_limit, fmt, d_err, stream) -> int:
        return load_library().kv_gather_latent(
            cache, scales, out, indices, index_dtype, index_stride, num_tokens, row_dim, out_dtype,
            None if strides is None else ctypes.byref(_LatentStrides(*strides)), page_size, size_limit,
            fmt, d_err, stream)

    @staticmethod
    def kv_attend_latent(q, out, lse, cache, scales, page_table, table_stride, table_width, seq_lens,
                         q_start, num_seqs, num_q_tokens, num_q_heads, row_dim, latent_dim, dtype,
                         strides: Optional[Sequence[int]], page_size, num_pages, fmt, sm_scale, work,
                         work_bytes, d_err, stream) -> int:
        return load_library().kv_attend_latent(
            q, out, lse, cache, scales, page_table, table_stride, table_width, seq_lens, q_start,
            num_seqs, num_q_tokens, num_q_heads, row_dim, latent_dim, dtype,
            None if strides is None else ctypes.byref(_AttendLatentStrides(*strides)), page_size,
            num_pages, fmt, sm_scale, work, work_bytes, d_err, stream)

    @staticmethod
    def kv_store_noalloc(k, v, k_cache, v_cache, indices, index_dtype, index_stride,
                         num_tokens, num_heads, head_dim, elem_bytes, strides: Sequence[int],
                         size_limit, num_split, stream):
        """kv_store without a caller-supplied error record (nothing is
        allocated; the record is a static array of the library). Blocks until
        the write is done; returns (status, oob_count, first_bad_token)."""
        st = _Strides(*[int(x) for x in strides])
        n = ctypes.c_int64(0)
        first = ctypes.c_int64(0)
        rc = load_library().kv_store_noalloc(k, v, k_cache, v_cache, indices, index_dtype,
                                             index_stride, num_tokens, num_heads, head_dim,
                                             elem_bytes, ctypes.byref(st), size_limit, num_split,
                                             ctypes.byref(n), ctypes.byref(first), stream)
        return rc, n.value, first.value

    @staticmethod
    def kv_error_poll(d_err, stream):
        n = ctypes.c_int64(0)
        first = ctypes.c_int64(0)
        rc = load_library().kv_error_poll(d_err, stream, ctypes.byref(n), ctypes.byref(first))
        return rc, n.value, first.value

    @staticmethod
    def kv_error_snapshot(d_err, dst, stream) -> int:
        return load_library().kv_error_snapshot(d_err, dst, stream)

    @staticmethod
    def kv_error_reset(d_err, stream) -> int:
        return load_library().kv_error_reset(d_err, stream)

    @staticmethod
    def kv_launch_floor(num_warps, stream) -> int:
        return load_library().kv_launch_floor(num_warps, stream)


# ---------------------------------------------------------------------------
# Tensor-level entry points
# ---------------------------------------------------------------------------

_default_records = {}


def error_record(device=None):
    """A zeroed device error record (two int64) owned by the caller."""
    import torch
    return torch.zeros(2, dtype=torch.int64, device=device or "cuda")


def _default_record(device):
    import torch
    dev = torch.device(device)
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    rec = _default_records.get(key)
    if rec is None:
        rec = _default_records[key] = error_record(torch.device("cuda", key))
    return rec


def _stream_handle(stream, device) -> int:
    if stream is None:
        import torch
        if device.index is not None:
            # the handle without a Stream object around it (2 us less)
            return torch._C._cuda_getCurrentRawStream(device.index)
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _rows3(x, H, D):
    """(token, head, dim) byte strides of a [T, H, D] or [T, H*D] tensor."""
    e = x.element_size()
    if x.dim() == 3:
        if tuple(x.shape[1:]) != (H, D):
            raise ValueError(f"row shape {tuple(x.shape)} != [T, {H}, {D}]")
        return x.stride(0) * e, x.stride(1) * e, x.stride(2) * e
    if x.dim() == 2:
        if x.shape[1] != H * D:
            raise ValueError(f"row width {x.shape[1]} != {H}*{D}")
        return x.stride(0) * e, D * x.stride(1) * e, x.stride(1) * e
    raise ValueError("rows must be 2-D or 3-D")


def _cache_shape(cache, num_heads=None, head_dim=None):
    """(slots, H, D) of a [slots, H, D] / [slots, H*D] / [pages, ps, H, D] cache."""
    if cache.dim() == 4:
        return cache.shape[0] * cache.shape[1], cache.shape[2], cache.shape[3]
    if cache.dim() == 3:
        return cache.shape[0], cache.shape[1], cache.shape[2]
    if cache.dim() == 2 and num_heads and head_dim:
        return cache.shape[0], num_heads, head_dim
    raise ValueError("cache must be [slots, H, D], [pages, page_size, H, D], or 2-D with "
                     "num_heads/head_dim given")


def _index_args(indices):
    import torch
    if indices.dim() != 1:
        raise ValueError("indices must be 1-D")
    if indices.dtype == torch.int32:
        return 0, indices.stride(0)
    if indices.dtype == torch.int64:
        return 1, indices.stride(0)
    raise TypeError("indices must be int32 or int64")


def _check(rc: int, what: str):
    if rc != KVStatus.OK:
        raise KVError(rc, what)


def kv_store(k, v, k_cache, v_cache, indices, *, size_limit: Optional[int] = None,
             num_split: int = 0, err=None, stream=None, num_heads: Optional[int] = None,
             head_dim: Optional[int] = None) -> None:
    """Plain copy of each token's K/V row into cache row ``indices[t]``.

    ``k``/``v``: [T, H, D] or [T, H*D] (any strides, any dtype); caches:
    [slots, H, D] or [slots, H*D] of the same element size. ``size_limit``
    defaults to the number of cache rows. Out-of-range slots are skipped and
    counted in ``err`` (a per-device default record if None); see
    :func:`kv_error_poll`.
    """
    slots, H, D = _cache_shape(k_cache, num_heads, head_dim)
    if k_cache.dim() == 4:
        raise ValueError("kv_store takes [slots, H, D] caches; use kv_store_fp8 for pages")
    e = k.element_size()
    if v.element_size() != e or k_cache.element_size() != e or v_cache.element_size() != e:
        raise TypeError("K, V and the caches must have the same element size")
    kt, kh, kd = _rows3(k, H, D)
    vt, vh, vd = _rows3(v, H, D)
    ks, khc, kdc = _rows3(k_cache, H, D)
    vs, vhc, vdc = _rows3(v_cache, H, D)
    idt, istride = _index_args(indices)
    T = indices.shape[0]
    if k.shape[0] < T or v.shape[0] < T:
        raise ValueError("fewer K/V rows than indices")
    rec = err if err is not None else _default_record(k.device)
    rc = raw.kv_store(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                      indices.data_ptr(), idt, istride, T, H, D, e,
                      (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc),
                      slots if size_limit is None else size_limit, num_split, rec.data_ptr(),
                      _stream_handle(stream, k.device))
    _check(rc, "kv_store")


def kv_store_fp8(k, v, k_cache, v_cache, indices, *, page_size: int = 1,
                 inv_k_scale=None, inv_v_scale=None, size_limit: Optional[int] = None,
                 err=None, stream=None, num_heads: Optional[int] = None,
                 head_dim: Optional[int] = None) -> None:
    """Fused scale + e4m3fn conversion + paged write.

    ``k``/``v``: bf16 or fp16 [T, H, D] or [T, H*D]. Caches: uint8 /
    float8_e4m3fn, [slots, H, D] (3-D) or [pages, page_size, H, D] (4-D).
    ``inv_k_scale``/``inv_v_scale``: fp32 device scalars (0-D or 1-element
    tensors); the scale is used only when both are given.
    """
    import torch
    slots, H, D = _cache_shape(k_cache, num_heads, head_dim)
    if k.dtype not in (torch.bfloat16, torch.float16) or v.dtype != k.dtype:
        raise TypeError("K and V must both be bf16 or both fp16")
    if k_cache.element_size() != 1 or v_cache.element_size() != 1:
        raise TypeError("FP8 caches have 1-byte elements")
    kt, kh, kd = _rows3(k, H, D)
    vt, vh, vd = _rows3(v, H, D)
    if k_cache.dim() == 4:
        if k_cache.shape[1] != page_size or v_cache.shape[1] != page_size:
            raise ValueError("page_size does not match the cache")
        kp, ks, khc, kdc = k_cache.stride()
        vp, vs, vhc, vdc = v_cache.stride()
    else:
        ks, khc, kdc = _rows3(k_cache, H, D)
        vs, vhc, vdc = _rows3(v_cache, H, D)
        kp, vp = ks * page_size, vs * page_size
    idt, istride = _index_args(indices)
    T = indices.shape[0]
    if k.shape[0] < T or v.shape[0] < T:
        raise ValueError("fewer K/V rows than indices")
    use_scale = int(inv_k_scale is not None and inv_v_scale is not None)
    for s in (inv_k_scale, inv_v_scale) if use_scale else ():
        if s.dtype != torch.float32 or s.numel() != 1 or s.device.type != "cuda":
            raise TypeError("inverse scales must be 1-element fp32 device tensors")
    rec = err if err is not None else _default_record(k.device)
    rc = raw.kv_store_fp8(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), indices.data_ptr(),
        idt, istride, T, H, D, 1 if k.dtype == torch.bfloat16 else 0,
        (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc), page_size, kp, vp,
        slots if size_limit is None else size_limit,
        inv_k_scale.data_ptr() if use_scale else None,
        inv_v_scale.data_ptr() if use_scale else None, use_scale, rec.data_ptr(),
        _stream_handle(stream, k.device))
    _check(rc, "kv_store_fp8")


def kv_error_poll(err=None, stream=None, device=None):
    """Synchronise, read and clear an error record: (status, oob_count, first_bad_token).

    ``KVStatus.ERR_WAIT``: a kernel of :func:`kv_attend` gave up a wait; its outputs are not to be used."""
    import torch
    if err is None:
        err = _default_record(device or torch.device("cuda", torch.cuda.current_device()))
    rc, n, first = raw.kv_error_poll(err.data_ptr(), _stream_handle(stream, err.device))
    if rc not in (KVStatus.OK, KVStatus.ERR_INDEX_OOB, KVStatus.ERR_WAIT):
        raise KVError(rc, "kv_error_poll")
    return KVStatus(rc), n, first


def kv_error_reset(err=None, stream=None, device=None) -> None:
    import torch
    if err is None:
        err = _default_record(device or torch.device("cuda", torch.cuda.current_device()))
    _check(raw.kv_error_reset(err.data_ptr(), _stream_handle(stream, err.device)),
           "kv_error_reset")


# ---------------------------------------------------------------------------
# Tensor-level wrappers of the other entry points
# ---------------------------------------------------------------------------

FP8_FORMATS = {"e4m3fn": 0, "e5m2": 1}
SCALE_MODES = {"none": 0, "tensor": 1, "token": 2, "token_head": 3, "page": 4}


def _paged_cache(cache, page_size, H, D):
    """(slot, head, dim, page) byte strides of a [slots, H, D] or [pages, ps, H, D] cache."""
    if cache.dim() == 4:
        if cache.shape[1] != page_size:
            raise ValueError("page_size does not match the cache")
        e = cache.element_size()
        sp, ss, sh, sd = (x * e for x in cache.stride())
        return ss, sh, sd, sp
    ss, sh, sd = _rows3(cache, H, D)
    return ss, sh, sd, ss * page_size


def _device_ptr_or_none(t):
    return None if t is None else t.data_ptr()


def kv_store_paged(k, v, k_cache, v_cache, indices, *, page_size: int, size_limit=None,
                   num_split: int = 0, err=None, stream=None) -> None:
    """Plain copy into [pages, page_size, H, D] caches (any page stride)."""
    slots, H, D = _cache_shape(k_cache)
    e = k.element_size()
    kt, kh, kd = _rows3(k, H, D)
    vt, vh, vd = _rows3(v, H, D)
    ks, khc, kdc, kp = _paged_cache(k_cache, page_size, H, D)
    vs, vhc, vdc, vp = _paged_cache(v_cache, page_size, H, D)
    idt, istride = _index_args(indices)
    rec = err if err is not None else _default_record(k.device)
    _check(raw.kv_store_paged(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                              indices.data_ptr(), idt, istride, indices.shape[0], H, D, e,
                              (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc), page_size, kp,
                              vp, slots if size_limit is None else size_limit, num_split,
                              rec.data_ptr(), _stream_handle(stream, k.device)), "kv_store_paged")


def kv_store_fp8_ex(k, v, k_cache, v_cache, indices, *, page_size: int = 1,
                    fmt: str = "e4m3fn", scale_mode: str = "none", inv_k_scale=None,
                    inv_v_scale=None, k_scales=None, v_scales=None, size_limit=None, err=None,
                    stream=None) -> None:
    """FP8 write in e4m3fn / e5m2 with no, per-tensor, per-token or per-(token, head)
    scales. Dynamic modes write the dequantisation scale of slot s (head h) to
    k_scales[s, h] / v_scales[s, h] (fp32 device tensors [slots, >= groups])."""
    slots, H, D = _cache_shape(k_cache)
    kt, kh, kd = _rows3(k, H, D)
    vt, vh, vd = _rows3(v, H, D)
    ks, khc, kdc, kp = _paged_cache(k_cache, page_size, H, D)
    vs, vhc, vdc, vp = _paged_cache(v_cache, page_size, H, D)
    idt, istride = _index_args(indices)
    sstride = 0
    if k_scales is not None:
        if k_scales.dim() != 2 or k_scales.stride(1) != 1 or v_scales.stride() != k_scales.stride():
            raise ValueError("scale caches must be [slots, groups] with unit inner stride")
        sstride = k_scales.stride(0)
    rec = err if err is not None else _default_record(k.device)
    import torch
    _check(raw.kv_store_fp8_ex(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), indices.data_ptr(),
        idt, istride, indices.shape[0], H, D, 1 if k.dtype == torch.bfloat16 else 0,
        (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc), page_size, kp, vp,
        slots if size_limit is None else size_limit, FP8_FORMATS[fmt], SCALE_MODES[scale_mode],
        _device_ptr_or_none(inv_k_scale), _device_ptr_or_none(inv_v_scale),
        _device_ptr_or_none(k_scales), _device_ptr_or_none(v_scales), sstride, rec.data_ptr(),
        _stream_handle(stream, k.device)), "kv_store_fp8_ex")


DYNAMIC_TENSOR_WORK_BYTES = 24  # KV_DYNAMIC_TENSOR_WORK_BYTES of the C header


def kv_store_fp8_dynamic_tensor(k, v, k_cache, v_cache, indices, *, page_size: int = 1,
                                fmt: str = "e4m3fn", scales=None, work=None, size_limit=None,
                                err=None, stream=None):
    """FP8 write with per-tensor scales formed from the batch, in one call:
    amax over all K (V) rows, inv = fmax / amax, codes fp8(x * inv).  Returns
    ``scales``: a 2-element fp32 device tensor receiving the forward scales
    amax / fmax (K, V).  ``work``: a device tensor of at least
    DYNAMIC_TENSOR_WORK_BYTES bytes, zero before its first use and reused
    across calls on one stream (a fresh zeroed one when None)."""
    import torch
    slots, H, D = _cache_shape(k_cache)
    kt, kh, kd = _rows3(k, H, D)
    vt, vh, vd = _rows3(v, H, D)
    ks, khc, kdc, kp = _paged_cache(k_cache, page_size, H, D)
    vs, vhc, vdc, vp = _paged_cache(v_cache, page_size, H, D)
    idt, istride = _index_args(indices)
    if k.dtype not in (torch.bfloat16, torch.float16) or v.dtype != k.dtype:
        raise TypeError("K and V must both be bf16 or both fp16")
    if scales is None:
        scales = torch.empty(2, dtype=torch.float32, device=k.device)
    if scales.dtype != torch.float32 or scales.numel() < 2 or not scales.is_contiguous():
        raise TypeError("scales must be a contiguous fp32 tensor of 2 elements")
    if work is None:
        work = torch.zeros(DYNAMIC_TENSOR_WORK_BYTES // 8, dtype=torch.int64, device=k.device)
    if work.numel() * work.element_size() < DYNAMIC_TENSOR_WORK_BYTES:
        raise ValueError(f"work holds fewer than {DYNAMIC_TENSOR_WORK_BYTES} bytes")
    rec = err if err is not None else _default_record(k.device)
    _check(raw.kv_store_fp8_dynamic_tensor(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), indices.data_ptr(),
        idt, istride, indices.shape[0], H, D, 1 if k.dtype == torch.bfloat16 else 0,
        (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc), page_size, kp, vp,
        slots if size_limit is None else size_limit, FP8_FORMATS[fmt], scales.data_ptr(),
        scales.data_ptr() + 4, work.data_ptr(), rec.data_ptr(), _stream_handle(stream, k.device)),
        "kv_store_fp8_dynamic_tensor")
    return scales


def kv_gather(k_cache, v_cache, k_out, v_out, indices, *, page_size: int = 1, size_limit=None,
              err=None, stream=None) -> None:
    """Row t of k_out / v_out takes the cache row of indices[t] (byte copy)."""
    slots, H, D = _cache_shape(k_cache)
    e = k_out.element_size()
    kt, kh, kd = _rows3(k_out, H, D)
    vt, vh, vd = _rows3(v_out, H, D)
    ks, khc, kdc, kp = _paged_cache(k_cache, page_size, H, D)
    vs, vhc, vdc, vp = _paged_cache(v_cache, page_size, H, D)
    idt, istride = _index_args(indices)
    rec = err if err is not None else _default_record(k_cache.device)
    _check(raw.kv_gather_paged(k_cache.data_ptr(), v_cache.data_ptr(), k_out.data_ptr(),
                               v_out.data_ptr(), indices.data_ptr(), idt, istride,
                               indices.shape[0], H, D, e,
                               (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc), page_size,
                               kp, vp, slots if size_limit is None else size_limit,
                               rec.data_ptr(), _stream_handle(stream, k_cache.device)),
           "kv_gather")


def kv_gather_fp8(k_cache, v_cache, k_out, v_out, indices, *, page_size: int = 1,
                  fmt: str = "e4m3fn", scale_mode: str = "none", k_scale=None, v_scale=None,
                  k_scales=None, v_scales=None, size_limit=None, err=None, stream=None) -> None:
    """Dequantising gather into bf16 / fp16 rows (the dtype of k_out)."""
    import torch
    slots, H, D = _cache_shape(k_cache)
    kt, kh, kd = _rows3(k_out, H, D)
    vt, vh, vd = _rows3(v_out, H, D)
    ks, khc, kdc, kp = _paged_cache(k_cache, page_size, H, D)
    vs, vhc, vdc, vp = _paged_cache(v_cache, page_size, H, D)
    idt, istride = _index_args(indices)
    sstride = k_scales.stride(0) if k_scales is not None else 0
    rec = err if err is not None else _default_record(k_cache.device)
    _check(raw.kv_gather_fp8_ex(
        k_cache.data_ptr(), v_cache.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
        indices.data_ptr(), idt, istride, indices.shape[0], H, D,
        1 if k_out.dtype == torch.bfloat16 else 0,
        (kt, kh, kd, vt, vh, vd, ks, khc, kdc, vs, vhc, vdc), page_size, kp, vp,
        slots if size_limit is None else size_limit, FP8_FORMATS[fmt], SCALE_MODES[scale_mode],
        _device_ptr_or_none(k_scale), _device_ptr_or_none(v_scale),
        _device_ptr_or_none(k_scales), _device_ptr_or_none(v_scales), sstride, rec.data_ptr(),
        _stream_handle(stream, k_cache.device)), "kv_gather_fp8")


def kv_inv_scale(scale, out=None, stream=None):
    """1 / scale in fp32 on the device; returns `out` (a new tensor if None)."""
    import torch
    if scale.dtype != torch.float32 or not scale.is_contiguous():
        raise TypeError("scale must be a contiguous fp32 tensor")
    out = torch.empty_like(scale) if out is None else out
    _check(raw.kv_inv_scale(scale.data_ptr(), out.data_ptr(), scale.numel(),
                            _stream_handle(stream, scale.device)), "kv_inv_scale")
    return out


def fused_fp8_set_kv_buffer(k, v, k_cache, v_cache, cache_loc, k_scale=None, v_scale=None,
                            page_size: int = 16, *, err=None, stream=None) -> None:
    """The fused FP8 write with the argument list of sglang trtllm_fp8_kv_kernel.py
    (`fused_fp8_set_kv_buffer`, its wrapper): K and V rows ([T, H, D] or
    [T, H*D], bf16 or fp16) go to slots ``cache_loc`` of e4m3fn caches,
    [slots, H, D] (``slots`` a multiple of ``page_size``) or
    [pages, page_size, H, D].  ``k_scale`` / ``v_scale`` are the forward
    (dequantisation) scales, Python floats or fp32 tensors, used only when both
    are given; as in that wrapper, ``1 / scale`` is formed on the device
    (``kv_inv_scale``), so tensor scales cost no host synchronisation.  The
    write itself is ``kv_store_fp8``; there is no second, unfused path.  The
    scale staging runs on ``stream`` (torch's current stream when None)."""
    import contextlib
    import torch
    if k_cache.dim() == 3 and k_cache.shape[0] % page_size:
        raise ValueError("cache slots must be a multiple of page_size")
    inv = None
    if k_scale is not None and v_scale is not None:
        ctx = (torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream)
               else contextlib.nullcontext())
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise TypeError("with scales, stream must be a torch.cuda.Stream or None")
        with ctx:
            sc = torch.empty(2, dtype=torch.float32, device=k.device)
            for i, x in enumerate((k_scale, v_scale)):
                if isinstance(x, torch.Tensor):
                    if x.numel() != 1:
                        raise ValueError("a scale tensor holds one value")
                    sc[i:i + 1].copy_(x.reshape(1))
                else:
                    sc[i:i + 1].fill_(float(x))
            inv = kv_inv_scale(sc, stream=stream)
    kv_store_fp8(k, v, k_cache, v_cache, cache_loc, page_size=page_size,
                 inv_k_scale=None if inv is None else inv[0:1],
                 inv_v_scale=None if inv is None else inv[1:2], err=err, stream=stream)


def kv_absmax_inv(k, v, *, fp8_max: float = 448.0, num_heads=None, head_dim=None, out=None,
                  work=None, stream=None):
    """Per-tensor max |K|, max |V| and fp8_max / amax on the device: returns a
    4-float tensor [amax_k, amax_v, inv_k, inv_v]. ``work``: an optional
    device workspace of at least 8 bytes, zero before first use, kept zero by
    the calls (two kernels per call instead of three)."""
    import torch
    if k.dim() == 3:
        H, D = k.shape[1], k.shape[2]
    else:
        H, D = num_heads, head_dim
    kt, kh, kd = _rows3(k, H, D)
    vt, vh, vd = _rows3(v, H, D)
    out = torch.empty(4, dtype=torch.float32, device=k.device) if out is None else out
    _check(raw.kv_absmax_inv(k.data_ptr(), v.data_ptr(), 1 if k.dtype == torch.bfloat16 else 0,
                             k.shape[0], H, D, (kt, kh, kd, vt, vh, vd, 0, 0, 0, 0, 0, 0), fp8_max,
                             out.data_ptr(), out.data_ptr() + 8,
                             None if work is None else work.data_ptr(),
                             _stream_handle(stream, k.device)),
           "kv_absmax_inv")
    return out


# ---------------------------------------------------------------------------
# The rotated append, the 4-bit cache and attention
# ---------------------------------------------------------------------------

CACHE_FORMATS = {None: 0, "e4m3fn": 1, "e2m1": 2}
ATTEND_WORK_BYTES = 64 << 20  # KV_ATTEND_WORK_BYTES of the C header
ATTEND_HEAD_BYTES = 256       # KV_ATTEND_HEAD_BYTES


def _is_bf16(dtype) -> int:
    import torch
    if dtype is torch.bfloat16:
        return 1
    if dtype is torch.float16:
        return 0
    raise TypeError("rows must be bf16 or fp16")


def _cache_strides(cache, page_size, width, elem_bytes, what):
    """(page, slot, head, dim) byte strides and the slots and heads of a
    [slots, H, width] or [pages, page_size, H, width] cache."""
    e = cache.element_size()
    if e != elem_bytes:
        raise TypeError(f"{what} must have {elem_bytes}-byte elements")
    if page_size < 1:
        raise ValueError("page_size must be at least 1")
    shape = cache.shape
    if len(shape) == 4:
        pages, ps, H, w = shape
        if ps != page_size:
            raise ValueError(f"page_size does not match {what}")
        page, slot, head, dim = cache.stride()
        slots = pages * ps
    elif len(shape) == 3:
        slots, H, w = shape
        slot, head, dim = cache.stride()
        page = slot * page_size
    else:
        raise ValueError(f"{what} must be [slots, H, {width}] or [pages, page_size, H, {width}]")
    if w != width:
        raise ValueError(f"{what}: rows of {w} elements, {width} expected")
    return page * e, slot * e, head * e, dim * e, slots, H


def _cache_pair(k_cache, v_cache, page_size, D, fmt, dtype):
    """The strides of both caches of format ``fmt`` (None: of ``dtype``)."""
    if fmt is None:
        if k_cache.dtype is not dtype or v_cache.dtype is not dtype:
            raise TypeError("without a format the caches have the rows' dtype")
        width, eb = D, 2
    else:
        width, eb = (D // 2 if fmt == "e2m1" else D), 1
    kc = _cache_strides(k_cache, page_size, width, eb, "k_cache")
    vc = _cache_strides(v_cache, page_size, width, eb, "v_cache")
    if kc[4:] != vc[4:]:
        raise ValueError("k_cache and v_cache differ in slots or heads")
    return kc, vc


def _block_scales(k_scales, v_scales, page_size, D, slots, H):
    if k_scales is None or v_scales is None:
        raise ValueError("an e2m1 cache needs k_scales and v_scales")
    out = [k_scales.data_ptr(), v_scales.data_ptr()]
    for x, what in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        page, slot, head, dim, n, h = _cache_strides(x, page_size, D // 16, 1, what)
        if dim != 1 or n != slots or h != H:
            raise ValueError(f"{what} must be [slots, H, D / 16] or [pages, page_size, H, D / 16] "
                             "bytes with contiguous rows, like the cache")
        out += (page, slot, head)
    return out


def _scalar_ptr(x, what):
    if x is None:
        return None
    import torch
    if x.dtype is not torch.float32 or x.numel() != 1 or not x.is_cuda:
        raise TypeError(f"{what} must be a 1-element fp32 device tensor")
    return x.data_ptr()


def _check_format(fmt):
    if fmt not in CACHE_FORMATS:
        raise ValueError(f"fmt must be one of {list(CACHE_FORMATS)}")
    return CACHE_FORMATS[fmt]


def kv_store_rope(k, v, k_cache, v_cache, indices, positions, cos_sin, *, q=None, q_out=None,
                  page_size: int = 1, interleaved: bool = False, fmt: Optional[str] = None,
                  inv_k_scale=None, inv_v_scale=None, k_scales=None, v_scales=None,
                  size_limit: Optional[int] = None, err=None, stream=None):
    """Append K/V rows to a cache with the position rotation applied on the way.

    ``k``/``v``: bf16 or fp16 [T, H, D]; ``q`` (optional): [T, HQ, D], rotated into ``q_out``
    (a new tensor on the caches' device if None; may be ``q``), which is returned. Token t goes
    to slot ``indices[t]`` at position ``positions[t]`` (1-D int32 / int64). ``cos_sin``: fp32
    [max_position, R], a row's R/2 cosines and then its sines; the first R dims of Q and K are
    rotated, in pairs (i, i + R/2), or (2i, 2i + 1) when ``interleaved``.

    ``fmt``: None (caches of the rows' dtype), "e4m3fn" (1-byte caches, [..., D]) or "e2m1"
    (uint8 caches [..., D / 2] with block scales ``k_scales`` / ``v_scales`` [..., D / 16]);
    caches and scales are [slots, H, ...] or [pages, page_size, H, ...]. ``inv_k_scale`` /
    ``inv_v_scale``: 1-element fp32 device tensors, the inverse tensor scales (None: 1).
    Tokens whose slot or position is out of range are skipped and counted in ``err``.
    """
    import torch
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or shape != v.shape or dtype is not v.dtype:
        raise ValueError("k and v must be [T, H, D] of one shape and dtype")
    T, H, D = shape
    bf16 = _is_bf16(dtype)
    f = _check_format(fmt)
    kc, vc = _cache_pair(k_cache, v_cache, page_size, D, fmt, dtype)
    if kc[5] != H:
        raise ValueError(f"caches of {kc[5]} heads, rows of {H}")
    if indices.shape != (T,) or positions.shape != (T,):
        raise ValueError("indices and positions must hold one entry per row")
    idt, istride = _index_args(indices)
    pdt, pstride = _index_args(positions)
    rows, rot = cos_sin.shape if cos_sin.dim() == 2 else (0, -1)
    tstride, tdim = cos_sin.stride() if rot >= 0 else (0, 0)
    if tdim != 1 or cos_sin.dtype is not torch.float32:
        raise TypeError("cos_sin must be fp32 [max_position, R] with contiguous rows")
    if q is not None:
        qshape = q.shape
        qst = q.stride()
        if len(qshape) != 3 or qshape[0] != T or qshape[2] != D or q.dtype is not dtype or qst[2] != 1:
            raise ValueError("q must be [T, HQ, D] of k's dtype with contiguous dims")
        if q_out is None:
            with _on_stream(stream, k_cache.device):  # (q itself may be page-locked host memory)
                q_out = torch.empty(qshape, dtype=dtype, device=k_cache.device)
        ost = q_out.stride()
        if q_out.shape != qshape or q_out.dtype is not dtype or ost[2] != 1:
            raise ValueError("q_out must be like q, with contiguous dims")
        qa = (q.data_ptr(), q_out.data_ptr(), qshape[1], qst[0] * 2, qst[1] * 2, ost[0] * 2, ost[1] * 2)
    elif q_out is not None:
        raise ValueError("q_out without q")
    else:
        qa = (None, None, 0, 0, 0, 0, 0)
    if fmt is None and not (inv_k_scale is None and inv_v_scale is None):
        raise ValueError("caches of the rows' dtype take no scales")
    sc = _block_scales(k_scales, v_scales, page_size, D, kc[4], H) if fmt == "e2m1" else None
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    device = k_cache.device
    rec = err if err is not None else _default_record(device)
    rc = raw.kv_store_rope(
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), indices.data_ptr(),
        idt, istride, T, H, D, bf16,
        (k0 * 2, k1 * 2, k2 * 2, v0 * 2, v1 * 2, v2 * 2, kc[1], kc[2], kc[3], vc[1], vc[2], vc[3]),
        page_size, kc[0], vc[0], kc[4] if size_limit is None else size_limit,
        (cos_sin.data_ptr(), tstride if rows > 1 else rot, rows, positions.data_ptr(), pdt, pstride,
         rot, 1 if interleaved else 0, *qa),
        f, _scalar_ptr(inv_k_scale, "inv_k_scale"), _scalar_ptr(inv_v_scale, "inv_v_scale"), sc,
        rec.data_ptr(), _stream_handle(stream, device))
    if rc:
        _check(rc, "kv_store_rope")
    return q_out


def kv_gather_fp4(k_cache, v_cache, k_scales, v_scales, k_out, v_out, indices, *,
                  page_size: int = 1, k_scale=None, v_scale=None, size_limit: Optional[int] = None,
                  err=None, stream=None) -> None:
    """Dequantising gather of an e2m1 cache (see :func:`kv_store_rope`) into bf16 / fp16 rows:
    row t of ``k_out`` / ``v_out`` [T, H, D] takes the cache row of ``indices[t]``.
    ``k_scale`` / ``v_scale``: the forward tensor scales (None: 1)."""
    shape = k_out.shape
    if len(shape) != 3 or shape != v_out.shape or k_out.dtype is not v_out.dtype:
        raise ValueError("k_out and v_out must be [T, H, D] of one shape and dtype")
    T, H, D = shape
    kc, vc = _cache_pair(k_cache, v_cache, page_size, D, "e2m1", None)
    if kc[5] != H:
        raise ValueError(f"caches of {kc[5]} heads, rows of {H}")
    sc = _block_scales(k_scales, v_scales, page_size, D, kc[4], H)
    idt, istride = _index_args(indices)
    n = indices.shape[0]
    if n > T:
        raise ValueError("fewer output rows than indices")
    k0, k1, k2 = k_out.stride()
    v0, v1, v2 = v_out.stride()
    device = k_cache.device
    rec = err if err is not None else _default_record(device)
    rc = raw.kv_gather_fp4(
        k_cache.data_ptr(), v_cache.data_ptr(), sc, k_out.data_ptr(), v_out.data_ptr(),
        indices.data_ptr(), idt, istride, n, H, D, _is_bf16(k_out.dtype),
        (k0 * 2, k1 * 2, k2 * 2, v0 * 2, v1 * 2, v2 * 2, kc[1], kc[2], kc[3], vc[1], vc[2], vc[3]),
        page_size, kc[0], vc[0], kc[4] if size_limit is None else size_limit,
        _scalar_ptr(k_scale, "k_scale"), _scalar_ptr(v_scale, "v_scale"), rec.data_ptr(),
        _stream_handle(stream, device))
    if rc:
        _check(rc, "kv_gather_fp4")


def _on_stream(stream, device):
    """The context in which torch allocates for `stream` (None: the current one)."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device)
    return torch.cuda.stream(stream)


def kv_attend(q, k_cache, v_cache, page_table, seq_lens, *, q_start=None, page_size=None,
              window: int = 0, sinks: int = 0, sm_scale: Optional[float] = None,
              fmt: Optional[str] = None, k_scale=None, v_scale=None, k_scales=None, v_scales=None,
              out=None, lse=None, work=None, err=None, stream=None):
    """Causal attention of ragged queries over a paged cache; returns ``out``.

    ``q``: bf16 or fp16 [tokens, HQ, D]. Caches as in :func:`kv_store_rope`
    ([pages, page_size, H, ...], or [slots, H, ...] with ``page_size`` given), HQ a multiple of
    H. ``page_table``: int32 [B, width] page ids; ``seq_lens``: int32 [B], the cached tokens of
    each sequence, its queries' own among them; ``q_start``: int32 [B + 1] offsets of each
    sequence's query rows, its newest tokens (None: one row per sequence).

    A query at position p sees key j <= p, with ``window`` > 0 only j > p - window or
    j < ``sinks``. ``sm_scale``: of the scores (1 / sqrt(D) if None). ``fmt``, ``k_scales``,
    ``v_scales``: as in :func:`kv_store_rope`; ``k_scale`` / ``v_scale``: forward tensor scales
    (1-element fp32 device tensors, None: 1). The same call gives the same bits; the rounding of
    a sequence's rows may differ with the others in the call, as the kernel is chosen for all
    (see the C header). ``lse``: an fp32 [tokens, HQ] tensor for the
    logarithms of the rows' sums, or None. ``work``: a device tensor that lets long sequences be
    split over the GPU (ATTEND_WORK_BYTES is always enough; its first ATTEND_HEAD_BYTES are zero
    before its first use, and every call that completes leaves them zero; calls that share one must
    not overlap; a new one per call if None). Sequences with a bad length or page id are counted in
    ``err``; a kernel that gave up a wait sets it to ``KVStatus.ERR_WAIT`` (see :func:`kv_error_poll`),
    and the outputs are not to be used.
    """
    import torch
    shape, dtype, qst = q.shape, q.dtype, q.stride()
    if len(shape) != 3 or qst[2] != 1:
        raise ValueError("q must be [tokens, HQ, D] with contiguous dims")
    T, HQ, D = shape
    bf16 = _is_bf16(dtype)
    f = _check_format(fmt)
    if page_size is None:
        if k_cache.dim() != 4:
            raise ValueError("page_size is needed with [slots, H, ...] caches")
        page_size = k_cache.shape[1]
    kc, vc = _cache_pair(k_cache, v_cache, page_size, D, fmt, dtype)
    if kc[3] != vc[3] or kc[3] != (2 if fmt is None else 1):
        raise ValueError("cache dims must be contiguous")
    slots, H = kc[4], kc[5]
    if H < 1 or HQ % H:
        raise ValueError(f"{HQ} query heads over {H} KV heads")
    sc = _block_scales(k_scales, v_scales, page_size, D, slots, H) if fmt == "e2m1" else None
    tst = page_table.stride()
    if len(tst) != 2 or page_table.dtype is not torch.int32 or tst[1] != 1:
        raise TypeError("page_table must be int32 [B, width] with contiguous rows")
    B, width = page_table.shape
    if seq_lens.dtype is not torch.int32 or seq_lens.shape != (B,) or (B > 1 and seq_lens.stride(0) != 1):
        raise TypeError("seq_lens must be a contiguous int32 [B]")
    if q_start is not None:
        if q_start.dtype is not torch.int32 or q_start.shape != (B + 1,) or q_start.stride(0) != 1:
            raise TypeError("q_start must be a contiguous int32 [B + 1]")
    elif T != B:
        raise ValueError("without q_start there is one query row per sequence")
    device = q.device
    if out is None:
        with _on_stream(stream, device):
            out = torch.empty(shape, dtype=dtype, device=device)
    ost = out.stride()
    if out.shape != shape or out.dtype is not dtype or ost[2] != 1:
        raise ValueError("out must be like q, with contiguous dims")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, HQ) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [tokens, HQ]")
    if work is None:
        with _on_stream(stream, device):
            work = torch.empty(ATTEND_WORK_BYTES, dtype=torch.uint8, device=device)
            work[:ATTEND_HEAD_BYTES].zero_()
    elif not work.is_contiguous():
        raise ValueError("work must be contiguous")
    rec = err if err is not None else _default_record(device)
    rc = raw.kv_attend(
        q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
        tst[0] if B > 1 else width, width, seq_lens.data_ptr(),
        None if q_start is None else q_start.data_ptr(), B, T, HQ, H, D, bf16,
        (qst[0] * 2, qst[1] * 2, ost[0] * 2, ost[1] * 2, kc[0], kc[1], kc[2], vc[0], vc[1], vc[2]),
        page_size, slots // page_size, f, _scalar_ptr(k_scale, "k_scale"),
        _scalar_ptr(v_scale, "v_scale"), sc, 1.0 / math.sqrt(D) if sm_scale is None else sm_scale,
        window, sinks, work.data_ptr(), work.numel() * work.element_size(), rec.data_ptr(),
        _stream_handle(stream, device))
    if rc:
        _check(rc, "kv_attend")
    return out


# ---------------------------------------------------------------------------
# A cache of latent rows
# ---------------------------------------------------------------------------

LATENT_FORMATS = {None: 0, "e4m3fn": 1}


def _latent_cache(cache, page_size, fmt, dtype):
    """(page, slot) byte strides, slots and row dims of a [slots, 1, D] or [pages, page_size, 1, D]
    cache of format ``fmt`` (None: of ``dtype``)."""
    if fmt not in LATENT_FORMATS:
        raise ValueError(f"fmt must be one of {list(LATENT_FORMATS)}")
    if fmt is None and cache.dtype is not dtype:
        raise TypeError("without a format the cache has the rows' dtype")
    shape = cache.shape
    D = shape[-1] if len(shape) else 0
    page, slot, _, dim, slots, H = _cache_strides(cache, page_size, D, 1 if fmt else 2, "cache")
    if H != 1 or (D > 1 and dim != (1 if fmt else 2)):
        raise ValueError("a latent cache has one head, with contiguous dims")
    return page, slot, slots, D


def _latent_scales(scales, fmt, slots):
    """(pointer, floats between slots) of the per-slot scales: [slots] or [slots, 1]."""
    if fmt is None:
        if scales is not None:
            raise ValueError("caches of the rows' dtype take no scales")
        return None, 1
    import torch
    if scales is None or scales.dtype is not torch.float32:
        raise TypeError("an e4m3fn cache needs fp32 scales")
    if scales.shape not in ((slots,), (slots, 1)):
        raise ValueError("scales must be [slots] or [slots, 1]")
    return scales.data_ptr(), scales.stride(0) if slots > 1 else 1


def kv_store_latent(c, r, cache, indices, positions=None, cos_sin=None, *, weight=None, eps: float = 1e-6,
                    q=None, q_out=None, page_size: int = 1, interleaved: bool = False,
                    fmt: Optional[str] = None, scales=None, size_limit: Optional[int] = None, err=None,
                    stream=None):
    """Form the latent rows of new tokens and write them to a cache of latent rows.

    ``c``: bf16 or fp16 [T, L], the latent dims; ``r``: [T, R] of the same dtype, the rotary dims
    (None: R = 0; both may be columns of one projection). With ``weight`` [L] the latent dims are
    divided by their root mean square (of which ``eps`` is added to the square) and multiplied by
    it. The first ``cos_sin.shape[1]`` rotary dims are rotated by ``positions[t]`` as in
    :func:`kv_store_rope`. ``q`` (optional): the rotary dims of the tokens' queries, [T, HQ, R],
    rotated into ``q_out`` (a new tensor on the cache's device if None; may be ``q``, or the rotary
    columns of whole query rows), which is returned.

    ``cache``: [slots, 1, L + R] or [pages, page_size, 1, L + R] with any slot and page strides.
    ``fmt``: None (the rows' dtype) or "e4m3fn" (1-byte elements; ``scales``: fp32 [slots] or
    [slots, 1], which takes each row's largest magnitude / 448). Tokens whose slot or position is
    out of range are skipped and counted in ``err``.
    """
    import torch
    dtype = c.dtype
    bf16 = _is_bf16(dtype)
    shape, st = c.shape, c.stride()
    if len(shape) != 2 or (shape[1] > 1 and st[1] != 1):
        raise ValueError("c must be [T, L] with contiguous dims")
    T, L = shape
    c_token, r_token = st[0] * 2, 0
    if r is None:
        R = 0
        if q is not None or positions is not None or cos_sin is not None:
            raise ValueError("positions, cos_sin and q belong to rotary dims (r)")
    else:
        shape, st = r.shape, r.stride()
        if len(shape) != 2 or shape[0] != T or r.dtype is not dtype or (shape[1] > 1 and st[1] != 1):
            raise ValueError("r must be [T, R] of c's dtype with contiguous dims")
        R, r_token = shape[1], st[0] * 2
        if positions is None or cos_sin is None:
            raise ValueError("rotary dims need positions and cos_sin")
    page, slot, slots, D = _latent_cache(cache, page_size, fmt, dtype)
    if D != L + R:
        raise ValueError(f"cache rows of {D} dims, {L} + {R} expected")
    if indices.shape != (T,):
        raise ValueError("indices must hold one entry per row")
    idt, istride = _index_args(indices)
    if weight is not None and (weight.dtype is not dtype or weight.shape != (L,) or not weight.is_contiguous()):
        raise ValueError("weight must be a contiguous [L] of c's dtype")
    sc, sc_slot = _latent_scales(scales, fmt, slots)
    device = cache.device
    rope = None
    if R:
        if positions.shape != (T,):
            raise ValueError("positions must hold one entry per row")
        pdt, pstride = _index_args(positions)
        rows, rot = cos_sin.shape if cos_sin.dim() == 2 else (0, -1)
        tstride, tdim = cos_sin.stride() if rot >= 0 else (0, 0)
        if (tdim != 1 and rot > 1) or rot < 0 or cos_sin.dtype is not torch.float32:
            raise TypeError("cos_sin must be fp32 [max_position, R] with contiguous rows")
        qa = (None, None, 0, 0, 0, 0, 0)
        if q is not None:
            shape, st = q.shape, q.stride()
            if len(shape) != 3 or shape[0] != T or shape[2] != R or q.dtype is not dtype or (R > 1 and st[2] != 1):
                raise ValueError("q must be [T, HQ, R] of c's dtype with contiguous dims")
            if q_out is None:
                with _on_stream(stream, device):  # (q itself may be page-locked host memory)
                    q_out = torch.empty(shape, dtype=dtype, device=device)
            so = st if q_out is q else q_out.stride()
            if q_out.shape != shape or q_out.dtype is not dtype or (R > 1 and so[2] != 1):
                raise ValueError("q_out must be like q, with contiguous dims")
            if shape[1]:
                qa = (q.data_ptr(), q_out.data_ptr(), shape[1], st[0] * 2, st[1] * 2, so[0] * 2, so[1] * 2)
        rope = (cos_sin.data_ptr(), tstride if rows > 1 else rot, rows, positions.data_ptr(), pdt, pstride, rot,
                1 if interleaved else 0, *qa)
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    rec = err if err is not None else _default_record(device)
    rc = raw.kv_store_latent(
        c.data_ptr(), r.data_ptr() if R else None, cache.data_ptr(), indices.data_ptr(), idt, istride, T, L, R, bf16,
        (c_token, r_token if R else 0, page, slot, sc_slot), page_size,
        slots if size_limit is None else size_limit, None if weight is None else weight.data_ptr(), eps, rope,
        LATENT_FORMATS[fmt], sc, rec.data_ptr(), _stream_handle(stream, device))
    if rc:
        _check(rc, "kv_store_latent")
    return q_out


def kv_gather_latent(cache, out, indices, *, page_size: int = 1, fmt: Optional[str] = None, scales=None,
                     size_limit: Optional[int] = None, err=None, stream=None) -> None:
    """Rows of a cache of latent rows (see :func:`kv_store_latent`) back: row t of ``out`` [T, L + R],
    bf16 or fp16, takes the row of ``indices[t]``, dequantised for "e4m3fn"."""
    shape, st = out.shape, out.stride()
    if len(shape) != 2 or (shape[1] > 1 and st[1] != 1):
        raise ValueError("out must be [T, L + R] with contiguous dims")
    bf16 = _is_bf16(out.dtype)
    page, slot, slots, D = _latent_cache(cache, page_size, fmt, out.dtype)
    if shape[1] != D:
        raise ValueError(f"cache rows of {D} dims, output rows of {shape[1]}")
    idt, istride = _index_args(indices)
    n = indices.shape[0]
    if n > shape[0]:
        raise ValueError("fewer output rows than indices")
    sc, sc_slot = _latent_scales(scales, fmt, slots)
    rec = err if err is not None else _default_record(cache.device)
    rc = raw.kv_gather_latent(cache.data_ptr(), sc, out.data_ptr(), indices.data_ptr(), idt, istride, n, D, bf16,
                              (st[0] * 2, 0, page, slot, sc_slot), page_size,
                              slots if size_limit is None else size_limit, LATENT_FORMATS[fmt], rec.data_ptr(),
                              _stream_handle(stream, cache.device))
    if rc:
        _check(rc, "kv_gather_latent")


def kv_attend_latent(q, cache, page_table, seq_lens, *, latent_dim: int, q_start=None, page_size=None,
                     sm_scale: Optional[float] = None, fmt: Optional[str] = None, scales=None, out=None, lse=None,
                     work=None, err=None, stream=None):
    """Causal attention of ragged queries over a paged cache of latent rows; returns ``out``.

    ``q``: bf16 or fp16 [tokens, HQ, D], D the cache rows' dims; ``out``: [tokens, HQ, latent_dim].
    Every head reads the same rows, whose first ``latent_dim`` dims are the values. ``cache``, ``fmt``
    and ``scales`` as in :func:`kv_store_latent` (``page_size`` is needed with a [slots, 1, D] cache);
    ``page_table``, ``seq_lens``, ``q_start``, ``lse``, ``work`` and ``err`` as in :func:`kv_attend`.
    ``sm_scale``: of the scores. Queries into which the keys' up-projection was multiplied still have their
    own head's products as scores: give 1 / sqrt(the dims, rotary ones included, of that head's queries and keys
    before it, 192 for 128 + 64). None is 1 / sqrt(D), which is right only where a head's queries are D dims of its own.
    """
    import torch
    dtype = q.dtype
    bf16 = _is_bf16(dtype)
    shape, sq = q.shape, q.stride()
    if len(shape) != 3 or (shape[2] > 1 and sq[2] != 1):
        raise ValueError("q must be [tokens, HQ, D] with contiguous dims")
    T, HQ, D = shape
    if page_size is None:
        if cache.dim() != 4:
            raise ValueError("page_size is needed with [slots, 1, D] caches")
        page_size = cache.shape[1]
    page, slot, slots, Dc = _latent_cache(cache, page_size, fmt, dtype)
    if Dc != D or not 1 <= latent_dim <= D:
        raise ValueError(f"queries of {D} dims, cache rows of {Dc}, {latent_dim} of them values")
    sc, sc_slot = _latent_scales(scales, fmt, slots)
    tst = page_table.stride()
    if len(tst) != 2 or page_table.dtype is not torch.int32 or tst[1] != 1:
        raise TypeError("page_table must be int32 [B, width] with contiguous rows")
    B, width = page_table.shape
    if seq_lens.dtype is not torch.int32 or seq_lens.shape != (B,) or (B > 1 and seq_lens.stride(0) != 1):
        raise TypeError("seq_lens must be a contiguous int32 [B]")
    if q_start is not None:
        if q_start.dtype is not torch.int32 or q_start.shape != (B + 1,) or q_start.stride(0) != 1:
            raise TypeError("q_start must be a contiguous int32 [B + 1]")
    elif T != B:
        raise ValueError("without q_start there is one query row per sequence")
    device = q.device
    shape = (T, HQ, latent_dim)
    if out is None:
        with _on_stream(stream, device):
            out = torch.empty(shape, dtype=dtype, device=device)
    so = out.stride()
    if out.shape != shape or out.dtype is not dtype or (latent_dim > 1 and so[2] != 1):
        raise ValueError("out must be [tokens, HQ, latent_dim] of q's dtype, with contiguous dims")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, HQ) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [tokens, HQ]")
    if work is None:
        with _on_stream(stream, device):
            work = torch.empty(ATTEND_WORK_BYTES, dtype=torch.uint8, device=device)
            work[:ATTEND_HEAD_BYTES].zero_()
    elif not work.is_contiguous():
        raise ValueError("work must be contiguous")
    rec = err if err is not None else _default_record(device)
    rc = raw.kv_attend_latent(
        q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), cache.data_ptr(), sc,
        page_table.data_ptr(), tst[0] if B > 1 else width, width, seq_lens.data_ptr(),
        None if q_start is None else q_start.data_ptr(), B, T, HQ, D, latent_dim, bf16,
        (sq[0] * 2, sq[1] * 2, so[0] * 2, so[1] * 2, page, slot, sc_slot), page_size,
        slots // page_size, LATENT_FORMATS[fmt], 1.0 / math.sqrt(D) if sm_scale is None else sm_scale, work.data_ptr(),
        work.numel() * work.element_size(), rec.data_ptr(), _stream_handle(stream, device))
    if rc:
        _check(rc, "kv_attend_latent")
    return out
