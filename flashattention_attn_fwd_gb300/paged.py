"""Python binding of the paged key/value cache (include/flattn.h): the cache
handle, the append of new tokens and the decode attention over it.  As in
``api`` only arguments are marshalled here; the library's kernels do the work.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _need
from ._lib import KV_FORMATS, MASKS, SCORE_MODS

_SCALE_BLOCK = 16


def _call_device(device: torch.device) -> None:
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _stream(stream, device: torch.device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _empty_on(stream, shape, dtype, device) -> torch.Tensor:
    """A tensor from the pool of the stream that the kernels run on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream),
                                           device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


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
        _same_device(k.device, v=v, k_scales=k_scales, v_scales=v_scales)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.format = "e2m1" if quantised else "bf16"
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.num_pages, self.page_size, self.Hkv, self.d = pages, page, Hkv, d
        self.device = k.device
        c = _lib.KvCache()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        if quantised:
            c.k_scales, c.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        c.k_scale, c.v_scale = self.k_scale, self.v_scale
        c.format = KV_FORMATS[self.format]
        c.num_pages, c.page_size, c.Hkv, c.d = pages, page, Hkv, d
        self._c = c
        self._ref = ctypes.byref(c)

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


def _need_table(cache, kv_len, block_table) -> int:
    """Checks the length and table arrays; returns B."""
    _need(kv_len, "kv_len", 1, torch.int32)
    _need(block_table, "block_table", 2, torch.int32)
    B = kv_len.shape[0]
    if not kv_len.is_contiguous():
        raise ValueError("kv_len must be contiguous")
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence of kv_len")
    if block_table.stride(1) != 1 and block_table.shape[1] > 1:
        raise ValueError("block_table must have contiguous rows")
    return B


def _rows(t, name, T, H, d):
    """Checks a [T, H, d] bf16 row tensor; returns its (token, head) strides."""
    _need(t, name, 3)
    if tuple(t.shape) != (T, H, d):
        raise ValueError(f"{name} must be {[T, H, d]}, got {list(t.shape)}")
    st, sh, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{name} must have a contiguous head dimension")
    # the stride of a single token or head is never used to step
    return (st if T > 1 else H * d, sh if H > 1 else d)


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
    B = _need_table(cache, kv_len, block_table)
    _need(k, "k", 3)
    T, Hkv, d = k.shape
    if Hkv != cache.Hkv or d != cache.d:
        raise ValueError(f"k must be [T, {cache.Hkv}, {cache.d}] for this cache, got {list(k.shape)}")
    a = _lib.KvAppendDesc()
    a.T, a.B, a.max_pages = T, B, block_table.shape[1]
    a.k_strides[:] = _rows(k, "k", T, Hkv, d)
    a.v_strides[:] = _rows(v, "v", T, Hkv, d)
    device = cache.device
    _call_device(device)
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", 1, torch.int32)
        if seq_offsets.shape[0] != B + 1 or not seq_offsets.is_contiguous():
            raise ValueError("seq_offsets must be contiguous [B + 1]")
        a.seq_offsets = seq_offsets.data_ptr()
    elif T != B:
        raise ValueError("without seq_offsets every sequence has one new token")
    if (rope_cos is None) != (rope_sin is None):
        raise ValueError("rope_cos and rope_sin come together")
    if rope_cos is not None:
        for name, t in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
            _need(t, name, 2, torch.float32)
            if not t.is_contiguous() or t.shape != rope_cos.shape:
                raise ValueError("rope_cos and rope_sin must be contiguous and of one shape")
        a.rope_cos, a.rope_sin = rope_cos.data_ptr(), rope_sin.data_ptr()
        a.rope_positions, a.rope_dim = rope_cos.shape[0], 2 * rope_cos.shape[1]
        a.rope_interleaved = 1 if rope_interleaved else 0
    if q is not None:
        _need(q, "q", 3)
        Hq = q.shape[1]
        if q_out is None:
            q_out = _empty_on(stream, (T, Hq, d), torch.bfloat16, device)
        a.Hq = Hq
        a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
        a.q_strides[:] = _rows(q, "q", T, Hq, d)
        a.q_out_strides[:] = _rows(q_out, "q_out", T, Hq, d)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out come together")
    if k_out is not None:
        a.k_out, a.v_out = k_out.data_ptr(), v_out.data_ptr()
        a.k_out_strides[:] = _rows(k_out, "k_out", T, Hkv, d)
        a.v_out_strides[:] = _rows(v_out, "v_out", T, Hkv, d)
    _same_device(device, k=k, v=v, kv_len=kv_len, block_table=block_table, seq_offsets=seq_offsets,
                 rope_cos=rope_cos, rope_sin=rope_sin, q=q, q_out=q_out, k_out=k_out, v_out=v_out)
    a.kv_len, a.block_table = kv_len.data_ptr(), block_table.data_ptr()
    a.table_stride = block_table.stride(0) if B > 1 else block_table.shape[1]
    a.stream = _stream(stream, device)
    st = _lib.lib().fl_kv_append(k.data_ptr(), v.data_ptr(), cache._ref, ctypes.byref(a))
    _lib.check(st, "fl_kv_append")
    return q_out


def _decode_desc(q, cache, block_table):
    _need(q, "q", 4)
    B, Hq, Lq, d = q.shape
    desc = _lib.AttnDesc()
    desc.B, desc.Hq, desc.Hkv, desc.Lq, desc.d, desc.dv = B, Hq, cache.Hkv, Lq, d, d
    desc.Lk = block_table.shape[1] * cache.page_size
    return desc


def _strides(t, name):
    """(b, h, l, c) strides; those of axes of length 1 are never used to step."""
    s, n = t.stride(), t.shape
    if s[3] != 1:
        raise ValueError(f"{name} must have a contiguous head dimension")
    full = (n[1] * n[2] * n[3], n[2] * n[3], n[3])
    return [x if m > 1 else f for x, m, f in zip(s, n, full)] + [1]


def attn_paged_decode_workspace_size(q, cache: PagedKVCache, block_table) -> int:
    """fl_attn_paged_decode_workspace_size: bytes of workspace that a call
    with these arguments needs."""
    _need(block_table, "block_table", 2, torch.int32)
    _call_device(cache.device)
    return int(_lib.lib().fl_attn_paged_decode_workspace_size(ctypes.byref(_decode_desc(q, cache, block_table)),
                                                              cache._ref))


def attn_paged_decode_fwd(q, cache: PagedKVCache, kv_len, block_table, *, mask: str = "none",
                          window: int | None = None, sink: int | None = None, score_mod: str = "none",
                          alibi_slopes=None, softcap: float | None = None, scale: float | None = None, out=None,
                          lse=None, return_lse: bool = True, workspace=None, stream=None):
    """fl_attn_paged_decode_fwd: q [B, Hq, Lq, d] bf16 (any strides that are
    multiples of 8) against the first kv_len[b] cached tokens of every
    sequence; mask "none", "causal" or "window" (with ``window`` and ``sink``).
    The workspace is allocated with torch when not given.  Returns (out
    [B, Hq, Lq, d] bf16, lse [B, Hq, Lq] fp32 or None)."""
    B = _need_table(cache, kv_len, block_table)
    desc = _decode_desc(q, cache, block_table)
    if q.shape[0] != B:
        raise ValueError("q must have one entry per sequence of kv_len")
    device = cache.device
    _call_device(device)
    if mask not in MASKS:
        raise ValueError(f"unknown mask {mask!r}")
    if score_mod not in SCORE_MODS:
        raise ValueError(f"unknown score_mod {score_mod!r}")
    desc.mask_kind, desc.score_mod = MASKS[mask], SCORE_MODS[score_mod]
    desc.window = 0 if window is None else int(window)
    desc.sink = 0 if sink is None else int(sink)
    desc.softcap = 0.0 if softcap is None else float(softcap)
    desc.scale = 0.0 if scale is None else float(scale)
    if alibi_slopes is not None:
        _need(alibi_slopes, "alibi_slopes", 1, torch.float32)
        if alibi_slopes.shape[0] != q.shape[1] or not alibi_slopes.is_contiguous():
            raise ValueError("alibi_slopes must be contiguous [Hq]")
        desc.alibi_slopes = alibi_slopes.data_ptr()
    if out is None:
        out = _empty_on(stream, q.shape, torch.bfloat16, device)
    else:
        _need(out, "out", 4)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is None and return_lse:
        lse = _empty_on(stream, q.shape[:3], torch.float32, device)
    elif lse is not None:
        _need(lse, "lse", 3, torch.float32)
        if lse.shape != q.shape[:3] or not lse.is_contiguous():
            raise ValueError("lse must be contiguous [B, Hq, Lq]")
    desc.q_strides[:] = _strides(q, "q")
    desc.o_strides[:] = _strides(out, "out")
    if workspace is None:
        n = int(_lib.lib().fl_attn_paged_decode_workspace_size(ctypes.byref(desc), cache._ref))
        workspace = _empty_on(stream, (max(n, 16),), torch.uint8, device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _same_device(device, q=q, kv_len=kv_len, block_table=block_table, alibi_slopes=alibi_slopes, out=out, lse=lse,
                 workspace=workspace)
    desc.stream = _stream(stream, device)
    st = _lib.lib().fl_attn_paged_decode_fwd(
        q.data_ptr(), cache._ref, kv_len.data_ptr(), block_table.data_ptr(),
        block_table.stride(0) if B > 1 else block_table.shape[1], out.data_ptr(),
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        ctypes.byref(desc))
    _lib.check(st, "fl_attn_paged_decode_fwd")
    return out, lse
