"""Chunks over the paged cache, its read-back and the rotary positions: the C
ABI's refusals, all of which return before any CUDA call (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

from flashattention_attn_fwd_gb300 import _lib
from tests.test_paged_abi import ALI, CACHES, INV, UNS, P, cache

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls with fake pointers stop at the missing GPU")
NAN, INF = float("nan"), float("inf")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from flashattention_attn_fwd_gb300.build import build
        build()
    return _lib.lib()


def fields(obj, base, kw):
    base.update(kw)
    for n, x in base.items():
        if n.endswith("_strides"):
            getattr(obj, n)[:] = x
        else:
            setattr(obj, n, x)
    return obj


# ------------------------------------------------------------------ prefill

def prefill_desc(**kw):
    return fields(_lib.new_desc(), dict(B=2, Hq=4, Hkv=2, Lq=5, Lk=64, d=64, dv=64, mask_kind=1), kw)


def prefill(L, c, d, q=P, off=P, n=P, table=P, stride=4, out=P, lse=P, ws=P, ws_bytes=1 << 40):
    return L.fl_attn_paged_prefill_fwd(q, ctypes.byref(c), off, n, table, stride, out, lse, ws, ws_bytes, ctypes.byref(d))


PREFILL = [
    (dict(B=0), INV), (dict(Lq=0), INV), (dict(Hq=3), INV), (dict(Hkv=4), INV), (dict(d=128), INV), (dict(dv=128), INV),
    (dict(Lk=65), INV), (dict(Lk=0), INV), (dict(Lq=2 ** 30 + 1), UNS), (dict(Lk=2 ** 30 + 16), UNS), (dict(Hq=258), UNS),
    (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(mask_kind=5), INV), (dict(mask_kind=-1), INV),
    (dict(mask_kind=3), UNS), (dict(mask_kind=4), UNS), (dict(mask_kind=2), INV), (dict(mask_kind=2, window=0), INV),
    (dict(mask_kind=2, window=3, sink=-1), INV), (dict(sink=1), INV), (dict(score_mod=3), INV), (dict(score_mod=1), INV),
    (dict(score_mod=2), INV), (dict(score_mod=2, softcap=INF), INV), (dict(score_mod=2, softcap=-1.0), INV),
    (dict(k_strides=(1, 1, 1, 1)), UNS), (dict(v_strides=(0, 0, 0, 1)), UNS),
    (dict(q_strides=(256, 64, 256, 1)), INV), (dict(q_strides=(0, 64, 256, 2)), INV), (dict(q_strides=(0, 32, 256, 1)), INV),
    (dict(q_strides=(0, 64, 32, 1)), INV), (dict(q_strides=(0, 68, 256, 1)), ALI), (dict(o_strides=(0, 64, 260, 1)), ALI),
    (dict(o_strides=(0, -64, 256, 1)), INV),
    (dict(score_mod=1, alibi_slopes=P + 2), ALI),
]


@pytest.mark.parametrize("kw,want", PREFILL, ids=str)
def test_prefill_refusals(L, kw, want):
    assert prefill(L, cache(), prefill_desc(**kw)) == want


@pytest.mark.parametrize("kw,want", CACHES, ids=str)
def test_prefill_and_read_refuse_bad_caches(L, kw, want):
    assert prefill(L, cache(**kw), prefill_desc(d=kw.get("d", 64), dv=kw.get("d", 64))) == want
    assert read(L, cache(**kw), read_desc()) == want


def test_prefill_pointers(L):
    c, d = cache(), prefill_desc()
    for kw in (dict(q=0), dict(n=0), dict(table=0), dict(out=0), dict(ws=0), dict(stride=3), dict(off=0)):
        assert prefill(L, c, d, **kw) == INV
    for kw in (dict(q=P + 8), dict(out=P + 8), dict(lse=P + 2), dict(off=P + 2), dict(n=P + 1), dict(table=P + 2),
               dict(ws=P + 8)):
        assert prefill(L, c, d, **kw) == ALI
    assert L.fl_attn_paged_prefill_fwd(P, 0, P, P, P, 4, P, P, P, 1 << 40, ctypes.byref(d)) == INV
    assert L.fl_attn_paged_prefill_fwd(P, ctypes.byref(c), P, P, P, 4, P, P, P, 1 << 40, 0) == INV
    assert L.fl_attn_paged_prefill_workspace_size(ctypes.byref(prefill_desc(B=0)), ctypes.byref(c)) == 0
    assert L.fl_attn_paged_prefill_workspace_size(0, ctypes.byref(c)) == 0


@no_gpu
def test_valid_calls_reach_the_device(L):
    """What passes every check fails on the missing GPU alone."""
    c4 = cache(format=1)
    for c in (cache(), c4):
        for kw in (dict(), dict(mask_kind=0), dict(mask_kind=2, window=7, sink=3), dict(score_mod=2, softcap=5.0),
                   dict(score_mod=1, alibi_slopes=P), dict(q_strides=(0, 64, 512, 1), o_strides=(0, 320, 64, 1)), dict(Hq=256)):
            assert prefill(L, c, prefill_desc(**kw)) == _lib.FL_ERR_CUDA, kw
        assert prefill(L, c, prefill_desc(Lq=2), off=0) == _lib.FL_ERR_CUDA
        assert prefill(L, c, prefill_desc(), lse=0) == _lib.FL_ERR_CUDA
        assert read(L, c, read_desc()) == _lib.FL_ERR_CUDA
    assert turn(L, rope_desc()) == _lib.FL_ERR_CUDA
    assert turn(L, rope_desc(Hk=0), k=0, ko=0) == _lib.FL_ERR_CUDA
    assert turn(L, rope_desc(), call="fl_rope_bwd") == _lib.FL_ERR_CUDA
    assert tables(L) == _lib.FL_ERR_CUDA


# --------------------------------------------------------------------- read

def read_desc(**kw):
    return fields(_lib.KvReadDesc(), dict(T=5, B=2, max_pages=4, seq_offsets=P, kv_len=P, block_table=P, table_stride=4,
                                          k_out_strides=(128, 64), v_out_strides=(128, 64)), kw)


def read(L, c, a, k=P, v=P):
    return L.fl_kv_read(ctypes.byref(c), k, v, ctypes.byref(a))


READ = [
    (dict(T=0), INV), (dict(B=0), INV), (dict(max_pages=0), INV), (dict(reserved0=1), INV), (dict(kv_len=0), INV),
    (dict(block_table=0), INV), (dict(table_stride=3), INV), (dict(seq_offsets=0), INV), (dict(max_pages=2 ** 27, table_stride=2 ** 27), UNS),
    (dict(k_out_strides=(128, 32)), INV), (dict(v_out_strides=(32, 64)), INV), (dict(k_out_strides=(132, 64)), ALI),
    (dict(kv_len=P + 2), ALI), (dict(block_table=P + 1), ALI), (dict(seq_offsets=P + 2), ALI),
]


@pytest.mark.parametrize("kw,want", READ, ids=str)
def test_read_refusals(L, kw, want):
    assert read(L, cache(), read_desc(**kw)) == want


def test_read_pointers(L):
    a = read_desc()
    assert read(L, cache(), a, k=0) == INV and read(L, cache(), a, v=0) == INV
    assert read(L, cache(), a, k=P + 8) == ALI and read(L, cache(), a, v=P + 8) == ALI
    assert L.fl_kv_read(0, P, P, ctypes.byref(a)) == INV
    assert L.fl_kv_read(ctypes.byref(cache()), P, P, 0) == INV


# --------------------------------------------------------------------- rope

def rope_desc(**kw):
    return fields(_lib.RopeDesc(), dict(B=2, L=5, Hq=4, Hk=2, d=64, rope_positions=64, rope_dim=64, rope_cos=P, rope_sin=P,
                                        positions=P, positions_stride=5), kw)


def turn(L, a, q=P, k=P, qo=P, ko=P, call="fl_rope_fwd"):
    return getattr(L, call)(q, k, qo, ko, ctypes.byref(a))


ROPE = [
    (dict(B=0), INV), (dict(L=0), INV), (dict(Hq=0), INV), (dict(Hk=0), INV), (dict(Hk=-1), INV), (dict(d=96), UNS),
    (dict(d=256), UNS), (dict(rope_cos=0), INV), (dict(rope_sin=0), INV), (dict(rope_positions=0), INV), (dict(rope_dim=0), INV),
    (dict(rope_dim=80), INV), (dict(rope_dim=24), UNS), (dict(rope_interleaved=2), INV), (dict(positions_stride=-1), INV),
    (dict(positions=0, L=65), INV), (dict(positions=P + 2), ALI), (dict(rope_cos=P + 8), ALI),
    (dict(q_strides=(0, 64, 64)), INV), (dict(q_strides=(64, 64, -64)), INV), (dict(k_strides=(64, 64, 68)), ALI),
    (dict(q_out_strides=(64, 68, 64)), ALI), (dict(k_out_strides=(64, 64, 0)), INV),
]


@pytest.mark.parametrize("call", ["fl_rope_fwd", "fl_rope_bwd"])
@pytest.mark.parametrize("kw,want", ROPE, ids=str)
def test_rope_refusals(L, kw, want, call):
    assert turn(L, rope_desc(**kw), call=call) == want


def test_rope_pointers(L):
    a = rope_desc()
    for kw in (dict(q=0), dict(qo=0), dict(k=0), dict(ko=0)):
        assert turn(L, a, **kw) == INV
    for kw in (dict(q=P + 8), dict(qo=P + 8), dict(k=P + 8), dict(ko=P + 8)):
        assert turn(L, a, **kw) == ALI
    assert L.fl_rope_fwd(P, P, P, P, 0) == INV


def tables(L, cos=P, sin=P, positions=64, rope_dim=64, **kw):
    s = fields(_lib.RopeScaling(), dict(base=1e4, factor=2.0, low_turns=1.0, high_turns=32.0, kind=0, original=64, amplitude=1.0), kw)
    return L.fl_rope_tables(cos, sin, positions, rope_dim, ctypes.byref(s), 0)


TABLES = [
    (dict(cos=0), INV), (dict(sin=0), INV), (dict(positions=0), INV), (dict(rope_dim=0), INV), (dict(rope_dim=24), UNS),
    (dict(rope_dim=144), UNS), (dict(cos=P + 8), ALI), (dict(sin=P + 4), ALI), (dict(base=1.0), INV), (dict(base=INF), INV),
    (dict(base=NAN), INV), (dict(kind=4), INV), (dict(kind=-1), INV), (dict(reserved=1), INV), (dict(amplitude=0.0), INV),
    (dict(amplitude=NAN), INV), (dict(kind=1, factor=0.5), INV), (dict(kind=2, factor=NAN), INV), (dict(kind=3, original=0), INV),
    (dict(kind=3, low_turns=-1.0), INV), (dict(kind=3, high_turns=1.0), INV), (dict(kind=3, high_turns=INF), INV),
]


@pytest.mark.parametrize("kw,want", TABLES, ids=str)
def test_table_refusals(L, kw, want):
    assert tables(L, **kw) == want


def test_tables_need_a_scaling(L):
    assert L.fl_rope_tables(P, P, 64, 64, 0, 0) == INV


def test_softcap_polynomial_is_the_forwards():
    """The chunk attention's host code states the forward's tanh polynomial."""
    csrc = os.path.join(ROOT, "flashattention_attn_fwd_gb300", "csrc")
    pat = re.compile(r"kTanh(?:Range|P\[4\]) = [^;]*;")
    texts = [sorted(set(pat.findall(open(os.path.join(csrc, f)).read()))) for f in ("api.cu", "paged_api.cu")]
    assert texts[0] and texts[0] == texts[1]


def test_python_checks():
    from flashattention_attn_fwd_gb300 import rope_fwd, rope_tables
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rope_fwd(x, None, torch.zeros(4, 32), torch.zeros(4, 32))
    with pytest.raises(ValueError):
        rope_tables(8, 64, scaling="square", device="cpu")


@pytest.mark.parametrize("axes", [(0, 1, 2), (0,), (1,), (2,), (1, 2)])
def test_rope_refuses_expanded_tensors(axes):
    """Three zero strides are the ABI's sign for contiguous: an expanded tensor
    must not get there."""
    from flashattention_attn_fwd_gb300 import rotary
    shape = (2, 3, 4, 64)
    x = torch.zeros([1 if i in axes else n for i, n in enumerate(shape)], dtype=torch.bfloat16).expand(shape)
    with pytest.raises(ValueError, match="expanded"):
        rotary._rows(x, "q", x.shape, x.get_device())
    assert rotary._rows(x.contiguous(), "q", x.shape, x.get_device()) == (768, 256, 64)


def test_rope_refuses_tables_that_want_a_gradient():
    from flashattention_attn_fwd_gb300 import rope
    x, t = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(4, 32, requires_grad=True)
    for cos, sin in ((t, t.detach()), (t.detach(), t)):
        with pytest.raises(ValueError, match="gradient"):
            rope(x, x, cos, sin)


def test_prefill_refuses_a_bf16_pool_past_its_row_count(L):
    """Groups of 8 rows of the pool and one page fit 31 bits, or the call is refused."""
    big, fits = 2 ** 34 // (2 * 16), 2 ** 34 // (2 * 16) - 2
    for fmt, pages, want in ((0, big, UNS), (0, 2 ** 31 - 1, UNS)):
        assert prefill(L, cache(format=fmt, num_pages=pages), prefill_desc()) == want
    if not torch.cuda.is_available():
        for fmt, pages in ((0, fits), (1, big)):
            assert prefill(L, cache(format=fmt, num_pages=pages), prefill_desc()) == _lib.FL_ERR_CUDA
