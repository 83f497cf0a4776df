"""Paged cache, append and paged decode: the C ABI's refusals, all of which
return before any CUDA call (no GPU)."""
import ctypes
import os

import pytest
import torch

from flashattention_attn_fwd_gb300 import _lib

P = 0x10000  # a 16-byte aligned fake device address; never dereferenced
INV, UNS, ALI = _lib.FL_ERR_INVALID_ARG, _lib.FL_ERR_UNSUPPORTED, _lib.FL_ERR_ALIGNMENT
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls with fake pointers stop at the missing GPU")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from flashattention_attn_fwd_gb300.build import build
        build()
    return _lib.lib()


def cache(**kw):
    c = _lib.KvCache()
    base = dict(k=P, v=P, k_scale=1.0, v_scale=1.0, format=0, num_pages=8, page_size=16, Hkv=2, d=64)
    if kw.get("format") == 1:
        base.update(k_scales=P, v_scales=P)
    base.update(kw)
    for n, x in base.items():
        setattr(c, n, x)
    return c


def append_desc(**kw):
    a = _lib.KvAppendDesc()
    base = dict(T=3, B=2, Hq=4, max_pages=4, seq_offsets=P, kv_len=P, block_table=P, table_stride=4, rope_cos=P,
                rope_sin=P, rope_positions=64, rope_dim=64, q=P, q_out=P)
    strides = dict(q_strides=(256, 64), k_strides=(128, 64), v_strides=(128, 64), q_out_strides=(256, 64),
                   k_out_strides=(128, 64), v_out_strides=(128, 64))
    base.update(strides)
    base.update(kw)
    for n, x in base.items():
        if n.endswith("_strides"):
            getattr(a, n)[:] = x
        else:
            setattr(a, n, x)
    return a


def append(L, c, a, k=P, v=P):
    return L.fl_kv_append(k, v, ctypes.byref(c), ctypes.byref(a))


CACHES = [
    (dict(k=0), INV), (dict(num_pages=0), INV), (dict(Hkv=0), INV), (dict(format=2), INV), (dict(format=-1), INV),
    (dict(k_scale=0.0, format=1), INV), (dict(v_scale=float("nan"), format=1), INV),
    (dict(k_scale=-1.0, format=1), INV), (dict(k_scale=float("inf"), format=1), INV),
    (dict(k_scale=1e-40, format=1), INV), (dict(k_scale=2.0), INV), (dict(k_scales=P), INV),
    (dict(format=1, v_scales=0), INV), (dict(d=32), UNS), (dict(d=96), UNS), (dict(page_size=24), UNS),
    (dict(page_size=8), UNS), (dict(page_size=512), UNS), (dict(Hkv=1 << 19), UNS), (dict(k=P + 8), ALI), (dict(format=1, k_scales=P + 4), ALI),
]


@pytest.mark.parametrize("kw,expect", CACHES)
def test_bad_cache_is_refused_by_both_calls(L, kw, expect):
    c = cache(**kw)
    assert append(L, c, append_desc()) == expect
    d = decode_desc(d=max(c.d, 1), dv=max(c.d, 1), Lk=max(4 * c.page_size, 1), Hkv=max(c.Hkv, 1), Hq=2 * max(c.Hkv, 1))
    assert decode(L, c, d) == expect
    assert L.fl_attn_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(c)) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(T=0), INV), (dict(B=0), INV), (dict(max_pages=0), INV), (dict(kv_len=0), INV), (dict(block_table=0), INV),
    (dict(table_stride=3), INV), (dict(seq_offsets=0), INV), (dict(rope_sin=0), INV), (dict(rope_positions=0), INV),
    (dict(rope_dim=0), INV), (dict(rope_dim=80), INV), (dict(rope_dim=24), UNS), (dict(rope_interleaved=2), INV),
    (dict(Hq=0), INV), (dict(q=0), INV), (dict(q_out=0), INV), (dict(Hq=3), INV), (dict(k_out=P), INV),
    (dict(v_out=P), INV), (dict(reserved0=1), INV), (dict(max_pages=1 << 27, table_stride=1 << 27), UNS),
    (dict(k_strides=(128, 68)), ALI), (dict(q_strides=(260, 64)), ALI), (dict(k_strides=(128, 32)), INV),
    (dict(q_out=P + 8), ALI), (dict(rope_cos=P + 4), ALI), (dict(kv_len=P + 2), ALI), (dict(block_table=P + 1), ALI),
    (dict(k_out=P, v_out=P, v_out_strides=(0, 0)), INV),
])
def test_append_refusals(L, kw, expect):
    assert append(L, cache(), append_desc(**kw)) == expect


def test_append_null_arguments(L):
    c, a = cache(), append_desc()
    assert append(L, c, a, k=0) == INV
    assert append(L, c, a, v=0) == INV
    assert append(L, c, a, v=P + 4) == ALI
    assert L.fl_kv_append(P, P, None, ctypes.byref(a)) == INV
    assert L.fl_kv_append(P, P, ctypes.byref(c), None) == INV


def decode_desc(**kw):
    d = _lib.new_desc()
    base = dict(B=2, Hq=4, Hkv=2, Lq=1, Lk=64, d=64, dv=64)
    base.update(kw)
    for n, x in base.items():
        setattr(d, n, x)
    return d


def decode(L, c, d, q=P, kv_len=P, table=P, stride=1 << 20, out=P, lse=0, ws=P, nbytes=1 << 40):
    return L.fl_attn_paged_decode_fwd(q, ctypes.byref(c), kv_len, table, stride, out, lse, ws, nbytes,
                                      ctypes.byref(d) if d is not None else None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), INV), (dict(Lq=0), INV), (dict(Hq=3), INV), (dict(Hkv=1, Hq=4), INV), (dict(d=128, dv=128), INV),
    (dict(dv=128), INV), (dict(Lk=70), INV), (dict(Hq=128, Lq=2), UNS),
    (dict(mask_kind=3), UNS), (dict(mask_kind=4), UNS), (dict(mask_kind=7), INV), (dict(mask_kind=2), INV),
    (dict(mask_kind=2, window=4, sink=-1), INV), (dict(mask_kind=1, sink=2), INV), (dict(sink=2), INV),
    (dict(score_mod=1), INV), (dict(score_mod=2), INV), (dict(score_mod=3), INV), (dict(scale=float("nan")), INV),
    (dict(B=1 << 30, Hq=64, Hkv=2), UNS),
])
def test_decode_refusals(L, kw, expect):
    assert decode(L, cache(), decode_desc(**kw)) == expect


@no_gpu
@pytest.mark.parametrize("kw", [dict(Lk=1 << 30, B=1), dict(mask_kind=2, window=4, sink=2)])
def test_decode_limits_accepted(L, kw):
    assert decode(L, cache(), decode_desc(**kw), stride=1 << 27) == _lib.FL_ERR_CUDA


def test_decode_pointers_and_strides(L):
    c = cache()
    for kw in (dict(q=0), dict(out=0), dict(kv_len=0), dict(table=0), dict(ws=0), dict(stride=3)):
        assert decode(L, c, decode_desc(), **kw) == INV, kw
    for kw in (dict(q=P + 8), dict(out=P + 2), dict(lse=P + 1), dict(kv_len=P + 2), dict(table=P + 1), dict(ws=P + 8)):
        assert decode(L, c, decode_desc(), **kw) == ALI, kw
    assert decode(L, c, None) == INV
    d = decode_desc()
    d.k_strides[:] = (1, 1, 1, 1)
    assert decode(L, c, d) == UNS
    d = decode_desc()
    d.q_strides[:] = (256, 64, 60, 1)
    assert decode(L, c, d) == ALI
    d.q_strides[:] = (256, 64, 64, 2)
    assert decode(L, c, d) == INV


def test_sink_belongs_to_the_window_mask(L):
    """Every entry point that takes an attention descriptor refuses sinks
    where its mask has none."""
    def desc(**kw):
        d = _lib.new_desc()
        base = dict(B=1, Hq=2, Hkv=2, Lq=128, Lk=128, d=64, dv=64)
        base.update(kw)
        for n, x in base.items():
            setattr(d, n, x)
        return d
    for kw in (dict(mask_kind=0, sink=1), dict(mask_kind=1, sink=1), dict(mask_kind=3, sink=1),
               dict(mask_kind=2, window=4, sink=-2)):
        d = desc(**kw)
        assert L.fl_attn_fwd(P, P, P, P, 0, ctypes.byref(d)) == INV, kw
        assert L.fl_attn_fwd_noalloc(P, P, P, P, 0, ctypes.byref(d)) == INV, kw
        assert L.fl_attn_bwd(P, P, P, P, P, P, P, P, P, P, 1 << 40, ctypes.byref(d)) == INV, kw
    d = desc(mask_kind=1, sink=1, Lq=1)
    assert L.fl_attn_decode_fwd(P, P, P, P, 0, 0, 0, 0, ctypes.byref(d)) == INV
    d = desc(mask_kind=1, sink=1, dv=128)
    assert L.fl_diffattn_fwd(P, P, P, P, P, P, 0, ctypes.c_float(0.5), ctypes.byref(d)) == INV


def test_python_layer_refuses_bad_tensors():
    from flashattention_attn_fwd_gb300 import PagedKVCache
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        PagedKVCache(k, k)            # not CUDA tensors
    with pytest.raises(ValueError):
        PagedKVCache.allocate(4, 16, 2, 64, format="int4", device="cpu")
    with pytest.raises(TypeError):
        PagedKVCache(None, k)


@pytest.mark.parametrize("kw", [dict(window=2 ** 31), dict(sink=2 ** 31), dict(Lk=-2 ** 31 - 1),
                                dict(q_strides=(2 ** 63, 1, 1, 1))], ids=str)
def test_values_past_the_descriptors_fields_are_refused(kw):
    """Not cut to the field's width: a ValueError before any call."""
    sizes = dict(B=1, Hq=1, Hkv=1, Lq=1, Lk=16, d=64, dv=64)
    rest = {k: v for k, v in kw.items() if k not in sizes}
    sizes.update({k: v for k, v in kw.items() if k in sizes})
    with pytest.raises(ValueError, match="range"):
        _lib.desc_pack(*sizes.values(), **rest)
