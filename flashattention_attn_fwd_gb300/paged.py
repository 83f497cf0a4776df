"""Python binding of the paged key/value cache (include/flattn.h): the cache
handle, the append of new tokens and the decode attention over it.  As in
``api`` only arguments are marshalled here; the library's kernels do the work.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _empty_on, _need, _raw_stream, _stream_ptr
from ._lib import KV_FORMATS, MASKS, SCORE_MODS

_SCALE_BLOCK = 16
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_Tensor = torch.Tensor
# the current device's index (CUDA is up: a cache on a device exists)
_device_index = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _check(t, name: str, ndim: int, dtype, index: int) -> None:
    """`t` is a tensor of this rank and type on CUDA device `index`."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.dim() != ndim or t.get_device() != index:
        _need(t, name, ndim, dtype)
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _current(index: int) -> None:
    if _device_index() != index:
        raise ValueError(f"the cache is on cuda:{index}, the current device is cuda:{_device_index()}")


class PagedKVCache:
    """fl_kv_cache: the page pool of a key/value cache, in bf16 or 4 bits.

    k, v      bf16 [num_pages, Hkv, page_size, d], or uint8
              [num_pages, Hkv, page_size, d / 2] (two e2m1 codes a byte)
    k_scales  uint8 (e4m3) [num_pages, Hkv, page_size, d / 16], 4-bit only
    v_scales  uint8 (e4m3) [num_pages, Hkv, d / 16, page_size], 4-bit only
    k_scale, v_scale  per-tensor scales of a 4-bit cache; a stored value is
              code * block scale * k_scale (v_scale)

    All contiguous, on one device.  ``allocate`` makes a zeroed pool.  Which
    page holds which tokens is the caller's block table."""

    def __init__(self, k, v, k_scales=None, v_scales=None, *, k_scale: float = 1.0, v_scale: float = 1.0):
        quantised = k_scales is not None or v_scales is not None
        for name, t in (("k", k), ("v", v)):
            _need(t, name, 4, torch.uint8 if quantised else torch.bfloat16)
        if k.shape != v.shape:
            raise ValueError("k and v must have the same shape")
        pages, Hkv, page, row = k.shape
        d = 2 * row if quantised else row
        if quantised:
            for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                _need(t, name, 4, torch.uint8)
            if tuple(k_scales.shape) != (pages, Hkv, page, d // _SCALE_BLOCK):
                raise ValueError("k_scales must be [num_pages, Hkv, page_size, d / 16]")
            if tuple(v_scales.shape) != (pages, Hkv, d // _SCALE_BLOCK, page):
                raise ValueError("v_scales must be [num_pages, Hkv, d / 16, page_size]")
        for name, t in (("k", k), ("v", v), ("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None and not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t is not None and t.device != k.device:
                raise ValueError(f"{name} must be on {k.device}, got {t.device}")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.format = "e2m1" if quantised else "bf16"
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.num_pages, self.page_size, self.Hkv, self.d = pages, page, Hkv, d
        self.device = k.device
        self.index = k.get_device()
        c = _lib.KvCache()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        if quantised:
            c.k_scales, c.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        c.k_scale, c.v_scale = self.k_scale, self.v_scale
        c.format = KV_FORMATS[self.format]
        c.num_pages, c.page_size, c.Hkv, c.d = pages, page, Hkv, d
        self._c = c
        self._ref = ctypes.addressof(c)

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, Hkv: int, d: int, *, format: str = "bf16",
                 k_scale: float = 1.0, v_scale: float = 1.0, device="cuda") -> "PagedKVCache":
        if format not in KV_FORMATS:
            raise ValueError(f"unknown cache format {format!r}")
        if format == "bf16":
            k, v = (torch.zeros((num_pages, Hkv, page_size, d), dtype=torch.bfloat16, device=device) for _ in range(2))
            return cls(k, v, k_scale=k_scale, v_scale=v_scale)
        k, v = (torch.zeros((num_pages, Hkv, page_size, d // 2), dtype=torch.uint8, device=device) for _ in range(2))
        ks = torch.zeros((num_pages, Hkv, page_size, d // _SCALE_BLOCK), dtype=torch.uint8, device=device)
        vs = torch.zeros((num_pages, Hkv, d // _SCALE_BLOCK, page_size), dtype=torch.uint8, device=device)
        return cls(k, v, ks, vs, k_scale=k_scale, v_scale=v_scale)


def _need_table(cache, kv_len, block_table) -> tuple[int, int, int]:
    """Checks the length and table arrays; returns (B, columns, row stride)."""
    _check(kv_len, "kv_len", 1, _I32, cache.index)
    _check(block_table, "block_table", 2, _I32, cache.index)
    B, n = block_table.shape
    if kv_len.numel() != B:
        raise ValueError("block_table must have one row per sequence of kv_len")
    if not kv_len.is_contiguous():
        raise ValueError("kv_len must be contiguous")
    row, col = block_table.stride()
    if col != 1 and n > 1:
        raise ValueError("block_table must have contiguous rows")
    return B, n, row if B > 1 else n


def _rows(t, name, T, H, d, index):
    """Checks a [T, H, d] bf16 row tensor; returns its (token, head) strides."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.get_device() != index or t.shape != (T, H, d):
        _check(t, name, 3, _BF16, index)
        raise ValueError(f"{name} must be {[T, H, d]}, got {list(t.shape)}")
    st, sh, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{name} must have a contiguous head dimension")
    # the stride of a single token or head is never used to step
    return (st if T > 1 else H * d), (sh if H > 1 else d)


def kv_append(cache: PagedKVCache, k, v, kv_len, block_table, *, seq_offsets=None, rope_cos=None, rope_sin=None,
              rope_interleaved: bool = False, q=None, q_out=None, k_out=None, v_out=None, stream=None):
    """fl_kv_append: rotate new tokens' q and k by their positions and append
    k and v to the cache.

    k, v [T, Hkv, d] and q [T, Hq, d] bf16 (any token and head strides that
    are multiples of 8); kv_len int32 [B] counts the new tokens; block_table
    int32 [B, max_pages]; seq_offsets int32 [B + 1] (None: one token per
    sequence); rope_cos, rope_sin fp32 [positions, rope_dim / 2] (None: no
    rotation).  q_out (allocated when q is given without it) takes the rotated
    queries; k_out and v_out, if given, the values that the cache now holds for
    the new tokens.  Returns q_out."""
    index = cache.index
    _current(index)
    B, max_pages, table_stride = _need_table(cache, kv_len, block_table)
    _check(k, "k", 3, _BF16, index)
    T, Hkv, d = k.shape
    if Hkv != cache.Hkv or d != cache.d:
        raise ValueError(f"k must be [T, {cache.Hkv}, {cache.d}] for this cache, got {list(k.shape)}")
    ks, vs = _rows(k, "k", T, Hkv, d, index), _rows(v, "v", T, Hkv, d, index)
    offsets = 0
    if seq_offsets is not None:
        _check(seq_offsets, "seq_offsets", 1, _I32, index)
        if seq_offsets.shape[0] != B + 1 or not seq_offsets.is_contiguous():
            raise ValueError("seq_offsets must be contiguous [B + 1]")
        offsets = seq_offsets.data_ptr()
    elif T != B:
        raise ValueError("without seq_offsets every sequence has one new token")
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("rope_cos and rope_sin come together")
    cos = sin = positions = rot = 0
    if rope_cos is not None:
        _check(rope_cos, "rope_cos", 2, _F32, index)
        _check(rope_sin, "rope_sin", 2, _F32, index)
        if rope_sin.shape != rope_cos.shape or not rope_cos.is_contiguous() or not rope_sin.is_contiguous():
            raise ValueError("rope_cos and rope_sin must be contiguous and of one shape")
        positions, rot = rope_cos.shape
        cos, sin, rot = rope_cos.data_ptr(), rope_sin.data_ptr(), 2 * rot
    Hq = qp = qop = 0
    qs = qos = kos = vos = (0, 0)
    if q is not None:
        _check(q, "q", 3, _BF16, index)
        Hq = q.shape[1]
        if q_out is None:
            q_out = _empty_on(stream, (T, Hq, d), _BF16, cache.device)
        qs, qos = _rows(q, "q", T, Hq, d, index), _rows(q_out, "q_out", T, Hq, d, index)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    kop = vop = 0
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out come together")
    if k_out is not None:
        kos, vos = _rows(k_out, "k_out", T, Hkv, d, index), _rows(v_out, "v_out", T, Hkv, d, index)
        kop, vop = k_out.data_ptr(), v_out.data_ptr()
    desc = _lib.APPEND_PACK(T, B, Hq, max_pages, offsets, kv_len.data_ptr(), block_table.data_ptr(), table_stride,
                            cos, sin, positions, rot, 1 if rope_interleaved else 0, 0, qp, qop, kop, vop,
                            *qs, *ks, *vs, *qos, *kos, *vos, _raw_stream(index) if stream is None else _stream_ptr(stream))
    st = _lib.lib().fl_kv_append(k.data_ptr(), v.data_ptr(), cache._ref, desc)
    if st:
        _lib.check(st, "fl_kv_append")
    return q_out


def _strides(t, name):
    """(b, h, l, c) strides; those of axes of length 1 are never used to step."""
    sb, sh, sl, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{name} must have a contiguous head dimension")
    B, H, L, d = t.shape
    return (sb if B > 1 else H * L * d, sh if H > 1 else L * d, sl if L > 1 else d, 1)


def attn_paged_decode_workspace_size(q, cache: PagedKVCache, block_table) -> int:
    """fl_attn_paged_decode_workspace_size: bytes of workspace that a call
    with these arguments needs."""
    _check(q, "q", 4, _BF16, cache.index)
    _check(block_table, "block_table", 2, _I32, cache.index)
    _current(cache.index)
    B, Hq, Lq, d = q.shape
    desc = _lib.desc_pack(B, Hq, cache.Hkv, Lq, block_table.shape[1] * cache.page_size, d, d)
    return int(_lib.lib().fl_attn_paged_decode_workspace_size(desc, cache._ref))


def attn_paged_decode_fwd(q, cache: PagedKVCache, kv_len, block_table, *, mask: str = "none",
                          window: int | None = None, sink: int | None = None, score_mod: str = "none",
                          alibi_slopes=None, softcap: float | None = None, scale: float | None = None, out=None,
                          lse=None, return_lse: bool = True, workspace=None, stream=None):
    """fl_attn_paged_decode_fwd: q [B, Hq, Lq, d] bf16 (any strides that are
    multiples of 8) against the first kv_len[b] cached tokens of every
    sequence; mask "none", "causal" or "window" (with ``window`` and ``sink``).
    The workspace is allocated with torch when not given.  Returns (out
    [B, Hq, Lq, d] bf16, lse [B, Hq, Lq] fp32 or None)."""
    index = cache.index
    _current(index)
    B, max_pages, table_stride = _need_table(cache, kv_len, block_table)
    _check(q, "q", 4, _BF16, index)
    shape = q.shape
    _, Hq, Lq, d = shape
    if shape[0] != B:
        raise ValueError("q must have one entry per sequence of kv_len")
    if mask not in MASKS:
        raise ValueError(f"unknown mask {mask!r}")
    if score_mod not in SCORE_MODS:
        raise ValueError(f"unknown score_mod {score_mod!r}")
    slopes = 0
    if alibi_slopes is not None:
        _check(alibi_slopes, "alibi_slopes", 1, _F32, index)
        if alibi_slopes.shape[0] != Hq or not alibi_slopes.is_contiguous():
            raise ValueError("alibi_slopes must be contiguous [Hq]")
        slopes = alibi_slopes.data_ptr()
    if out is None:
        out = _empty_on(stream, shape, _BF16, cache.device)
    else:
        _check(out, "out", 4, _BF16, index)
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    if lse is None and return_lse:
        lse = _empty_on(stream, shape[:3], _F32, cache.device)
    elif lse is not None:
        _check(lse, "lse", 3, _F32, index)
        if lse.shape != shape[:3] or not lse.is_contiguous():
            raise ValueError("lse must be contiguous [B, Hq, Lq]")
    desc = _lib.desc_pack(B, Hq, cache.Hkv, Lq, max_pages * cache.page_size, d, d, scale=scale or 0.0,
                          mask_kind=MASKS[mask], window=window or 0, sink=sink or 0, score_mod=SCORE_MODS[score_mod],
                          softcap=softcap or 0.0, slopes=slopes, q_strides=_strides(q, "q"),
                          o_strides=_strides(out, "out"),
                          stream=_raw_stream(index) if stream is None else _stream_ptr(stream))
    L = _lib.lib()
    if workspace is None:
        n = int(L.fl_attn_paged_decode_workspace_size(desc, cache._ref))
        workspace = _empty_on(stream, (max(n, 16),), torch.uint8, cache.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{index}")
    st = L.fl_attn_paged_decode_fwd(q.data_ptr(), cache._ref, kv_len.data_ptr(), block_table.data_ptr(), table_stride,
                                    out.data_ptr(), 0 if lse is None else lse.data_ptr(), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), desc)
    if st:
        _lib.check(st, "fl_attn_paged_decode_fwd")
    return out, lse
