"""GPU tests of reading the paged cache back: bit for bit the stored rows (bf16)
or code * block scale * cache scale in 32 bits, rounded once more to bf16."""
import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import FlattnError, PagedKVCache, kv_append, kv_read, sync_status, synth
from tests._paged import pool, rope_tables, table_for, unpack
from tests.test_gpu_paged import DEV, dev, make_cache

pytestmark = pytest.mark.gpu


def expected(cache, lens, new, table, T):
    """(k, v) [T, Hkv, d] fp32 of the rows that are written, and which are."""
    K, V, codes = unpack(cache)
    page = cache.page_size
    if codes is not None:  # the two products' roundings, in 32 bits
        kc, vc, ks, vs = codes
        K = (oracle.dequantise(kc, ks, 1.0).astype(np.float32) * np.float32(cache.k_scale)).astype(np.float32)
        V = (oracle.dequantise(vc, vs, 1.0).astype(np.float32) * np.float32(cache.v_scale)).astype(np.float32)
    k = np.full((T, cache.Hkv, cache.d), 7.0, np.float32)
    v, t = k.copy(), 0
    for b, n in enumerate(new):
        for i in range(n):
            pos = lens[b] - n + i
            if pos >= 0:
                k[t + i], v[t + i] = K[table[b, pos // page], :, pos % page], V[table[b, pos // page], :, pos % page]
        t += n
    return torch.from_numpy(k).bfloat16(), torch.from_numpy(v).bfloat16()


CASES = [
    # Hkv, d, page, lens, rows
    (1, 64, 16, [1], [1]),
    (3, 128, 32, [40, 7, 0, 33], [40, 3, 0, 1]),
    (8, 64, 64, [701], [701]),
    (2, 128, 256, [513, 300], [257, 299]),
    (4, 64, 16, [5, 20], [9, 20]),     # rows at negative positions are left
    (5, 128, 16, [100] * 40, [3] * 40),
]


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rows_come_back_bit_for_bit(case, fmt):
    Hkv, d, page, lens, rows = case
    pages = sum(-(-n // page) for n in lens) + 2
    parts, _, _ = pool(fmt, pages, Hkv, page, d, seed=page)
    cache = make_cache(parts, **(dict(k_scale=0.77, v_scale=1.3) if fmt == "e2m1" else {}))
    table = table_for(lens, page, pages, seed=3)
    T = sum(rows) + 2  # two rows behind the last sequence
    off = dev([0] + list(np.cumsum(rows)), torch.int32)
    ko, vo = (torch.full((T, Hkv, d), 7.0, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k, v = kv_read(cache, dev(lens, torch.int32), dev(table), T, seq_offsets=off, k_out=ko, v_out=vo)
    sync_status()
    assert k is ko and v is vo
    ek, ev = expected(cache, lens, rows, table, T)
    assert torch.equal(k.cpu(), ek) and torch.equal(v.cpu(), ev)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_without_offsets_strides_and_another_stream(fmt):
    B, Hkv, d, page = 37, 3, 64, 16
    lens = [(11 * b) % 50 + 1 for b in range(B)]
    pages = sum(-(-n // page) for n in lens)
    parts, _, _ = pool(fmt, pages, Hkv, page, d, seed=1)
    cache = make_cache(parts)
    table = table_for(lens, page, pages, seed=2)
    wide = np.full((B, table.shape[1] + 3), 10 ** 8, np.int32)
    wide[:, :table.shape[1]] = table
    room = torch.full((B, 2 * Hkv + 1, 2 * d), 7.0, device=DEV, dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = dev(lens, torch.int32), dev(wide)[:, :table.shape[1]]
    torch.cuda.synchronize()
    kv_read(cache, *args, B, k_out=room[:, :Hkv, :d], v_out=room[:, Hkv:2 * Hkv, :d], stream=s)
    s.synchronize()
    sync_status()
    ek, ev = expected(cache, lens, [1] * B, table, B)
    assert torch.equal(room[:, :Hkv, :d].cpu(), ek) and torch.equal(room[:, Hkv:2 * Hkv, :d].cpu(), ev)
    assert (room[:, :, d:] == 7).all() and (room[:, 2 * Hkv] == 7).all()
    k, v = kv_read(cache, *args, B)
    sync_status()
    assert torch.equal(k.cpu(), ek) and torch.equal(v.cpu(), ev)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_what_was_appended_comes_back_as_the_append_gave_it(fmt):
    Hkv, d, page, new = 2, 128, 32, [50, 1, 90]
    x = synth.randn_bf16((sum(new), 2 * Hkv, d), synth.generator(4)).to(DEV)
    cache = PagedKVCache.allocate(16, page, Hkv, d, format=fmt, **(dict(k_scale=0.5, v_scale=2.0) if fmt == "e2m1" else {}))
    table = dev(table_for(new, page, 16, seed=1))
    off, n = dev([0, 50, 51, 141], torch.int32), dev(new, torch.int32)
    cos, sin = (t.to(DEV) for t in rope_tables(100, 64))
    ko, vo = (torch.empty((sum(new), Hkv, d), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    kv_append(cache, x[:, :Hkv], x[:, Hkv:], n, table, seq_offsets=off, rope_cos=cos, rope_sin=sin, k_out=ko, v_out=vo)
    k, v = kv_read(cache, n, table, sum(new), seq_offsets=off)
    sync_status()
    assert torch.equal(k, ko) and torch.equal(v, vo)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_bad_pages_are_left_and_reported(fmt):
    lens, page = [60, 64], 16
    parts, _, _ = pool(fmt, 16, 2, page, 64, seed=7)
    cache = make_cache(parts)
    table = table_for(lens, page, 16, seed=5)
    off, n = dev([0, 60, 124], torch.int32), dev(lens, torch.int32)
    ek, ev = expected(cache, lens, lens, table, 124)
    ek[32:48], ev[32:48] = 7.0, 7.0
    for bad in (-1, 16, 2 ** 31 - 1, -2 ** 31):
        t2 = table.copy()
        t2[0, 2] = bad
        ko, vo = (torch.full((124, 2, 64), 7.0, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        kv_read(cache, n, dev(t2), 124, seq_offsets=off, k_out=ko, v_out=vo)
        with pytest.raises(FlattnError) as e:
            sync_status()
        assert e.value.status == 6
        assert torch.equal(ko.cpu(), ek) and torch.equal(vo.cpu(), ev)
    # a length past the table: the rows with a column come, the others are left
    ko, vo = (torch.full((124, 2, 64), 7.0, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    kv_read(cache, dev([60, 74], torch.int32), dev(table), 124, seq_offsets=off, k_out=ko, v_out=vo)
    with pytest.raises(FlattnError):
        sync_status()
    ek, ev = expected(cache, lens, lens, table, 124)
    assert torch.equal(ko[:60].cpu(), ek[:60]) and (ko[114:] == 7).all()
    assert torch.equal(ko[60:114].cpu(), ek[70:]) and torch.equal(vo[60:114].cpu(), ev[70:])
