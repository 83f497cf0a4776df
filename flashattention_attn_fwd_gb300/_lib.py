"""ctypes view of the C ABI declared in include/flattn.h.

This module only loads ``libflattn.so`` and mirrors its types; it performs no
computation.  The library must have been built (``__graft_entry__.build()``
or ``python -m flashattention_attn_fwd_gb300.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflattn.so")

FL_OK = 0
FL_ERR_INVALID_ARG = 1
FL_ERR_UNSUPPORTED = 2
FL_ERR_ALIGNMENT = 3
FL_ERR_CUDA = 4
FL_ERR_TIMEOUT = 5
FL_ERR_DEVICE_BOUNDS = 6

MASKS = {"none": 0, "causal": 1, "window": 2, "prefix_lm": 3, "document": 4}
SCORE_MODS = {"none": 0, "alibi": 1, "softcap": 2}
FL_DEBUG_SKIP_KV_LOAD = 0x1
FL_DEBUG_KEY_SPLIT = 0x2

# Every symbol include/flattn.h declares.
EXPORTS = (
    "fl_attn_desc_init",
    "fl_attn_fwd",
    "fl_diffattn_fwd",
    "fl_evoformer_gated_attn_fwd",
    "fl_evoformer_col_gated_attn_fwd",
    "fl_sync_status",
    "fl_status_string",
    "fl_abi_version",
    "fl_attn_desc_size",
    "fl_attn_fwd_noalloc",
    "fl_attn_decode_fwd",
    "fl_attn_decode_workspace_size",
    "fl_attn_bwd",
    "fl_attn_bwd_workspace_size",
    "fl_diffattn_bwd",
    "fl_diffattn_bwd_workspace_size",
    "fl_last_error_detail",
    "fl_attn_schedule",
    "fl_kv_append",
    "fl_attn_paged_decode_fwd",
    "fl_attn_paged_decode_workspace_size",
    "fl_kv_cache_size",
    "fl_kv_append_desc_size",
)

KV_FORMATS = {"bf16": 0, "e2m1": 1}


class AttnDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("Lq", ctypes.c_int32), ("Lk", ctypes.c_int32), ("d", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("mask_kind", ctypes.c_int32), ("doc_causal", ctypes.c_int32),
        ("window", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
        ("score_mod", ctypes.c_int32), ("softcap", ctypes.c_float),
        ("alibi_slopes", ctypes.c_void_p), ("doc_offsets", ctypes.c_void_p),
        ("num_docs", ctypes.c_int32),
        ("q_strides", ctypes.c_int64 * 4), ("k_strides", ctypes.c_int64 * 4),
        ("v_strides", ctypes.c_int64 * 4), ("o_strides", ctypes.c_int64 * 4),
        ("stream", ctypes.c_void_p),
        ("debug_flags", ctypes.c_uint32), ("debug_arg", ctypes.c_int32),
        ("wait_limit_ms", ctypes.c_uint32),
        ("sink", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 6),
    ]


class KvCache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("format", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 5),
    ]


class KvAppendDesc(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("seq_offsets", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("rope_cos", ctypes.c_void_p), ("rope_sin", ctypes.c_void_p),
        ("rope_positions", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
        ("rope_interleaved", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p),
        ("q_strides", ctypes.c_int64 * 2), ("k_strides", ctypes.c_int64 * 2), ("v_strides", ctypes.c_int64 * 2),
        ("q_out_strides", ctypes.c_int64 * 2), ("k_out_strides", ctypes.c_int64 * 2),
        ("v_out_strides", ctypes.c_int64 * 2),
        ("stream", ctypes.c_void_p),
    ]


# The structures as one packed bytes object (native alignment): a fraction of
# the time of setting ctypes fields one by one.
_ATTN = struct.Struct("@7i f 5i f 2P i 16q P I i I i 6i")
_APPEND = struct.Struct("@4i 3P q 2P 4i 4P 12q P")
_ZERO4 = (0, 0, 0, 0)


def _packer(layout: struct.Struct):
    def pack(*values):
        try:
            return layout.pack(*values)
        except struct.error as e:
            raise ValueError(f"argument out of the descriptor's range: {e}") from None
    return pack


APPEND_PACK = _packer(_APPEND)
ATTN_PACK = _packer(_ATTN)


def desc_pack(B, Hq, Hkv, Lq, Lk, d, dv, *, scale=0.0, mask_kind=0, doc_causal=0, window=0, prefix=0, score_mod=0,
              softcap=0.0, slopes=0, doc_offsets=0, num_docs=0, q_strides=_ZERO4, k_strides=_ZERO4,
              v_strides=_ZERO4, o_strides=_ZERO4, stream=0, debug_flags=0, debug_arg=-1, wait_limit_ms=0, sink=0):
    """fl_attn_desc as bytes."""
    return ATTN_PACK(B, Hq, Hkv, Lq, Lk, d, dv, scale, mask_kind, doc_causal, window, prefix, score_mod, softcap,
                     slopes, doc_offsets, num_docs, *q_strides, *k_strides, *v_strides, *o_strides, stream,
                     debug_flags, debug_arg, wait_limit_ms, sink, 0, 0, 0, 0, 0, 0)


class FlattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status == FL_ERR_CUDA:
            detail = lib().fl_last_error_detail().decode()
        super().__init__(f"{what}: {status_string(status)} (status {status})" + (f" [{detail}]" if detail else ""))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                "(the CUDA library is required; there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        # structures are passed as pointers, ctypes.byref(...) or packed bytes
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        L.fl_attn_desc_init.argtypes = [ctypes.POINTER(AttnDesc)]
        L.fl_attn_desc_init.restype = None
        L.fl_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp]
        L.fl_attn_fwd.restype = i32
        L.fl_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp]
        L.fl_attn_fwd_noalloc.restype = i32
        L.fl_diffattn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, vp]
        L.fl_diffattn_fwd.restype = i32
        L.fl_evoformer_gated_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp]
        L.fl_evoformer_gated_attn_fwd.restype = i32
        L.fl_evoformer_col_gated_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp]
        L.fl_evoformer_col_gated_attn_fwd.restype = i32
        L.fl_attn_decode_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.fl_attn_decode_fwd.restype = i32
        L.fl_attn_decode_workspace_size.argtypes = [vp]
        L.fl_attn_decode_workspace_size.restype = ctypes.c_size_t
        L.fl_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.fl_attn_bwd.restype = i32
        L.fl_attn_bwd_workspace_size.argtypes = [vp]
        L.fl_attn_bwd_workspace_size.restype = ctypes.c_size_t
        L.fl_diffattn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp,
                                      ctypes.c_size_t, vp]
        L.fl_diffattn_bwd.restype = i32
        L.fl_diffattn_bwd_workspace_size.argtypes = [vp]
        L.fl_diffattn_bwd_workspace_size.restype = ctypes.c_size_t
        L.fl_sync_status.argtypes = [vp]
        L.fl_sync_status.restype = i32
        L.fl_attn_schedule.argtypes = [ctypes.POINTER(AttnDesc), vp, ctypes.POINTER(ctypes.c_int64)]
        L.fl_attn_schedule.restype = i32
        L.fl_last_error_detail.argtypes = []
        L.fl_last_error_detail.restype = ctypes.c_char_p
        L.fl_status_string.argtypes = [i32]
        L.fl_status_string.restype = ctypes.c_char_p
        L.fl_abi_version.argtypes = []
        L.fl_abi_version.restype = i32
        L.fl_kv_append.argtypes = [vp, vp, vp, vp]
        L.fl_kv_append.restype = i32
        L.fl_attn_paged_decode_fwd.argtypes = [vp, vp, vp, vp, ctypes.c_int64, vp, vp, vp,
                                               ctypes.c_size_t, vp]
        L.fl_attn_paged_decode_fwd.restype = i32
        L.fl_attn_paged_decode_workspace_size.argtypes = [vp, vp]
        L.fl_attn_paged_decode_workspace_size.restype = ctypes.c_size_t
        L.fl_kv_cache_size.argtypes = []
        L.fl_kv_cache_size.restype = i32
        L.fl_kv_append_desc_size.argtypes = []
        L.fl_kv_append_desc_size.restype = i32
        L.fl_attn_desc_size.argtypes = []
        L.fl_attn_desc_size.restype = i32
        if L.fl_attn_desc_size() != ctypes.sizeof(AttnDesc) or ctypes.sizeof(AttnDesc) != _ATTN.size:
            raise RuntimeError("fl_attn_desc layout mismatch between flattn.h and the binding")
        if L.fl_kv_cache_size() != ctypes.sizeof(KvCache) or \
                L.fl_kv_append_desc_size() != ctypes.sizeof(KvAppendDesc) or \
                ctypes.sizeof(KvAppendDesc) != _APPEND.size:
            raise RuntimeError("paged cache layout mismatch between flattn.h and the binding")
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fl_status_string(int(status)).decode()


def new_desc() -> AttnDesc:
    d = AttnDesc()
    lib().fl_attn_desc_init(ctypes.byref(d))
    return d


def check(status: int, what: str) -> None:
    if status != FL_OK:
        raise FlattnError(status, what)
