"""GPU tests of attention of chunks of new tokens over the paged cache, against
the 64-bit oracle with bounds derived per element.

Bound.  As for the paged decode (tests/test_gpu_paged.py): each weight carries
its score's error ds (relative) and the rounding of P, half a step of its type
(bf16 2^-8, fp16 2^-11), so that out is off by at most (2 ds + rP) sum_j P_j |v_j|,
then rounded to bf16: 2^-8 |out|.  ds: (d + 8) 2^-24 mag + 2^-21, a 4-bit cache's
query 2^-25 top more.  Softcap: a polynomial within 6.2e-7 of tanh, relative, where
|tanh| < 0.47 (3e-7 cap), else 1 - 2 / (1 + e^2y) with an exponential and a
reciprocal of 2^-22 each: below 2^-20 cap.  P is taken against a reference at most
the row's maximum, so the largest weight is at least 1 (2^7 in fp16) and what is
too small for P's type is at most 2^-126 (bf16) or 2^-32 (fp16) of it; weights
up to 2^8 of the reference fit both types.  Pieces joined in 32 bits add a few
2^-24, below the 2 % taken for products of errors.
"""
import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import (FlattnError, attn_fwd, attn_paged_decode_fwd, attn_paged_prefill_fwd,
                                           attn_paged_prefill_workspace_size, sync_status, synth)
from tests._paged import pool, table_for
from tests.test_gpu_paged import DEV, dev, make_cache

pytestmark = pytest.mark.gpu


def reference(q, K, V, lens, new, table, **kw):
    """The oracle sequence by sequence: (out [T, Hq, d], lse [T, Hq], and the
    bounds' parts in the same layout)."""
    parts, t = [], 0
    for b, n in enumerate(new):
        if n:
            qb = q[t:t + n].transpose(0, 1)[None]
            r = oracle.paged_attention(qb, K, V, lens[b:b + 1], np.maximum(table[b:b + 1], 0), **kw)
            parts.append([np.swapaxes(x[0], 0, 1) for x in r])
        t += n
    return [np.concatenate([p[i] for p in parts]) for i in range(6)]


def check(out, lse, ref, fmt, d, cap=0.0):
    ro, rl, amp, tot, mag, top = ref
    n = ro.shape[0]
    ds = ((d + 8) * 2.0 ** -24 * mag + 2.0 ** -21 + 2.0 ** -20 * cap)[..., None]
    if fmt == "e2m1":
        ds = ds + 2.0 ** -25 * top[..., None]
    rp = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -11
    lost = 2.0 ** -126 if fmt == "bf16" else 2.0 ** -32
    got = out[:n].double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = 1.02 * ((2 * ds + rp) * amp + 2.0 ** -8 * np.abs(ro) + lost * tot)
    err = np.abs(got - ro)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:5].tolist())
    if lse is not None:
        gl = lse[:n].double().cpu().numpy()
        live = np.isfinite(rl)
        assert np.array_equal(live, np.isfinite(gl)) and (gl[~live] == -np.inf).all()
        assert (np.abs(gl[live] - rl[live]) <= (2 * ds[..., 0] + 2.0 ** -20)[live] + 2.0 ** -22 * np.abs(rl[live])).all()


def setup(fmt, Hq, Hkv, d, page, past, new, seed, spare=3, pages=None, width=None):
    lens = [p + n for p, n in zip(past, new)]
    pages = sum(-(-max(n, 0) // page) for n in lens) + spare if pages is None else pages
    scales = dict(k_scale=0.75, v_scale=1.5) if fmt == "e2m1" else {}
    parts, K, V = pool(fmt, pages, Hkv, page, d, seed=seed, **scales)
    table = table_for([max(n, 0) for n in lens], page, pages, seed=seed + 1, width=width)
    q = synth.randn_bf16((sum(new), Hq, d), synth.generator(seed + 2))
    if fmt == "e2m1":
        q = (q.float() * 0.2).bfloat16()  # scales reach 448: scores of ordinary size
    off = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    return parts, scales, K, V, table, q, lens, off


CASES = [
    # Hq, Hkv, d, page, past, new, kwargs
    (1, 1, 64, 16, [0], [1], {}),
    (1, 1, 128, 16, [0], [1], {}),
    (4, 2, 64, 16, [5], [3], {}),
    (8, 2, 128, 32, [0, 40, 0], [33, 1, 70], {}),
    (8, 2, 64, 64, [100, 0, 7], [0, 129, 64], {}),
    (2, 2, 64, 128, [130, 3], [300, 257], {}),
    (2, 2, 128, 256, [255, 0], [131, 513], {}),
    (6, 2, 64, 16, [300, 0], [50, 43], {}),              # groups of 3: 126 rows a slot
    (5, 1, 128, 32, [128, 100], [27, 28], {}),
    (7, 1, 64, 64, [500], [19], dict(mask="none")),
    (128, 1, 64, 16, [60], [3], {}),                      # a token a slot
    (100, 1, 128, 32, [33], [2], {}),
    (8, 1, 128, 16, [200, 17], [40, 16], dict(mask="none")),
    (8, 2, 64, 32, [900, 40, 0], [100, 30, 1], dict(mask="window", window=100, sink=4)),
    (4, 2, 128, 16, [700, 3], [200, 90], dict(mask="window", window=33, sink=150)),
    (4, 1, 128, 64, [300], [260], dict(mask="window", window=1, sink=0)),
    (4, 1, 64, 128, [300, 60], [61, 10], dict(mask="window", window=1 << 30, sink=200)),
    (8, 2, 64, 32, [300, 90], [70, 20], dict(score_mod="softcap", softcap=5.0)),
    (8, 2, 128, 32, [300, 90], [70, 20], dict(score_mod="softcap", softcap=30.0, scale=0.3)),
    (4, 1, 128, 16, [30], [140], dict(score_mod="softcap", softcap=1e5, mask="window", window=50, sink=3)),
    (8, 2, 128, 32, [300, 0], [70, 200], dict(score_mod="alibi")),
    (6, 2, 64, 16, [300, 0], [70, 200], dict(score_mod="alibi", mask="window", window=64, sink=1)),
]


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:4]) + "-" + "_".join(map(str, c[5])) +
                         "-" + "-".join(f"{a}{b}" for a, b in c[6].items()))
def test_against_the_oracle(case, fmt):
    Hq, Hkv, d, page, past, new, kw = case
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=d + page)
    kw = dict(mask="causal", **kw) if "mask" not in kw else kw
    okw, gkw = dict(kw), dict(kw)
    if kw.get("score_mod") == "alibi":
        s = synth.alibi_slopes(Hq)
        okw["slopes"], gkw["alibi_slopes"] = s.numpy(), s.to(DEV)
    ref = reference(q, K, V, lens, new, table, **okw)
    out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table),
                                      seq_offsets=dev(off), **gkw)
    sync_status()
    check(out, lse, ref, fmt, d, kw.get("softcap", 0.0))


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
def test_units_that_many_blocks_share_and_blocks_with_many_units(fmt, d):
    """A few tokens over a long past (every unit cut into many pieces) beside
    sequences of all lengths, and only short ones (many units a block)."""
    for past, new in (([9000, 0, 3, 500], [5, 40, 1, 300]), ([0] * 90, [(5 * b) % 37 for b in range(90)])):
        Hq, Hkv, page = 4, 2, 16
        parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=5)
        ref = reference(q, K, V, lens, new, table, mask="causal")
        out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table),
                                          seq_offsets=dev(off))
        sync_status()
        check(out, lse, ref, fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_more_sequences_than_threads(fmt):
    """B = 1100, zero to three tokens each, one row a sequence without offsets."""
    B, Hq, Hkv, d, page = 1100, 2, 1, 64, 16
    new = [(b * 7) % 4 for b in range(B)]
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, [(3 * b) % 40 for b in range(B)], new, seed=6)
    cache = make_cache(parts, **scales)
    out, lse = attn_paged_prefill_fwd(q.to(DEV), cache, dev(lens, torch.int32), dev(table), seq_offsets=dev(off))
    sync_status()
    check(out, lse, reference(q, K, V, lens, new, table, mask="causal"), fmt, d)
    out, lse = attn_paged_prefill_fwd(q[:B].to(DEV), cache, dev(lens, torch.int32), dev(table))
    sync_status()
    check(out, lse, reference(q[:B], K, V, lens, [1] * B, table, mask="causal"), fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("page", [16, 256])
def test_ignores_what_no_row_sees(fmt, page):
    """Stale NaNs and infinities behind the last token and between sinks and
    window, and missing pages, change nothing."""
    Hq, Hkv, d = 4, 2, 64
    past, new, kw = [423, 900], [20, 3], dict(mask="window", window=40, sink=5)
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=7)
    ref = reference(q, K, V, lens, new, table, **kw)
    parts = [t.clone() if t is not None else None for t in parts]
    t2 = table.copy()
    for b, n in enumerate(lens):
        seen = set(range(5)) | set(range(n - new[b] - 40 + 1, n))
        for c in range(-(-n // page)):
            if not seen & set(range(c * page, (c + 1) * page)):
                t2[b, c] = (-1, 10 ** 6)[b]
        for j in range(-(-n // page) * page):
            if j not in seen:
                pg, at = table[b, j // page], j % page
                if fmt == "bf16":
                    parts[0][pg, :, at] = float("nan")
                    parts[1][pg, :, at] = float("inf") if j & 1 else float("nan")
                else:
                    parts[2][pg, :, at] = 0x7f      # e4m3 NaN
                    parts[3][pg, :, :, at] = 0xff
    out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(t2),
                                      seq_offsets=dev(off), **kw)
    sync_status()
    check(out, lse, ref, fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("page", [16, 128])
def test_a_bad_page_is_left_out_and_reported(fmt, page):
    """Keys of a page outside the pool count for nothing; the other sequence
    and the next call are right."""
    Hq, Hkv, d = 4, 2, 64
    past, new = [300, 64], [30, 20]
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=8)
    cache, n, o = make_cache(parts, **scales), dev(lens, torch.int32), dev(off)
    pages = parts[0].shape[0]
    ref = reference(q, K, V, lens, new, table, mask="causal")
    # sequence 0 without the page: its other pages' keys as a sequence of their own
    # (the page lies before every row, so that causal sees the same of them)
    rest = reference(q[:new[0]], K, V, [lens[0] - page], new[:1], np.delete(table[:1], 1, axis=1), mask="causal")
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t2 = table.copy()
        t2[0, 1] = bad
        out, lse = attn_paged_prefill_fwd(q.to(DEV), cache, n, dev(t2), seq_offsets=o)
        with pytest.raises(FlattnError) as e:
            sync_status()
        assert e.value.status == 6
        check(out[new[0]:], lse[new[0]:], [x[new[0]:] for x in ref], fmt, d)
        check(out[:new[0]], lse[:new[0]], rest, fmt, d)
    out, lse = attn_paged_prefill_fwd(q.to(DEV), cache, n, dev(table), seq_offsets=o)
    sync_status()
    check(out, lse, ref, fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_every_number_outside_the_pool_is_a_bad_page(fmt):
    """-2 and others next to the pool's limits are left out and reported alike."""
    past, new = [96], [16]
    parts, scales, K, V, table, q, lens, off = setup(fmt, 4, 2, 64, 16, past, new, seed=14)
    cache, n, o = make_cache(parts, **scales), dev(lens, torch.int32), dev(off)
    pages = parts[0].shape[0]
    rest = reference(q, K, V, [lens[0] - 16], new, np.delete(table, 2, axis=1), mask="causal")
    for bad in (-2, -3, -2 ** 31 + 1, pages, pages + 1):
        t2 = table.copy()
        t2[0, 2] = bad
        out, lse = attn_paged_prefill_fwd(q.to(DEV), cache, n, dev(t2), seq_offsets=o)
        with pytest.raises(FlattnError) as e:
            sync_status()
        assert e.value.status == 6
        check(out, lse, rest, fmt, 64)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_lengths_and_offsets_at_their_limits(fmt):
    """Lengths past the table are clamped, below zero nothing is seen; more new
    rows than tokens: those at negative positions see nothing; rows behind the
    last sequence are left as they are."""
    Hq, Hkv, d, page = 2, 1, 64, 16
    scales = dict(k_scale=0.75, v_scale=1.5) if fmt == "e2m1" else {}
    parts, K, V = pool(fmt, 8, Hkv, page, d, seed=9, **scales)
    table = np.array([[3, 1], [5, 0], [2, 7], [4, 6]], np.int32)
    new, lens = [2, 3, 9, 0], [10 ** 9, -5, 4, 7]
    T = sum(new)
    q = (synth.randn_bf16((T + 4, Hq, d), synth.generator(3)).float() * 0.2).bfloat16()
    off = dev([0] + list(np.cumsum(new)), torch.int32)
    out = torch.full((T + 4, Hq, d), 7.0, device=DEV, dtype=torch.bfloat16)
    lse = torch.full((T + 4, Hq), 7.0, device=DEV)
    for mask in ("causal", "none"):
        attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table), seq_offsets=off,
                               mask=mask, out=out, lse=lse)
        sync_status()
        ref = reference(q[:T], K, V, [32, 0, 4, 7], new, table, mask=mask)
        check(out, lse, ref, fmt, d)
        assert (out[2:5] == 0).all() and (lse[2:5] == -float("inf")).all()
        if mask == "causal":
            assert (out[5:10] == 0).all() and (lse[5:10] == -float("inf")).all()
        assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    # no sequence has a row
    zero = torch.zeros(5, device=DEV, dtype=torch.int32)
    out.fill_(7.0)
    attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table), seq_offsets=zero, out=out)
    sync_status()
    assert (out == 7).all()


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_strides_streams_workspace_graph_and_repeatability(fmt):
    """Head-major q and out, a table with padded rows, a workspace with a guard,
    two calls at once on two streams, a captured call replayed with other
    lengths; the same call gives the same bits."""
    Hq, Hkv, d, page = 8, 2, 128, 32
    past, new = [1500, 0, 37], [100, 260, 1]
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=10)
    cache, n, o = make_cache(parts, **scales), dev(lens, torch.int32), dev(off)
    T = sum(new)
    padded = np.full((3, table.shape[1] + 5), 10 ** 7, np.int32)
    padded[:, :table.shape[1]] = table
    tab = dev(padded)[:, :table.shape[1]]
    room = torch.full((Hq + 1, T, d + 8), 7.0, device=DEV, dtype=torch.bfloat16)
    qs = torch.zeros((Hq, T, d + 8), device=DEV, dtype=torch.bfloat16)
    qs[:, :, :d] = q.to(DEV).transpose(0, 1)
    qv, ov = qs[:, :, :d].transpose(0, 1), room[:Hq, :, :d].transpose(0, 1)
    need = attn_paged_prefill_workspace_size(qv, cache, tab)
    ws = [torch.full((need + 256,), 0xA5, device=DEV, dtype=torch.uint8) for _ in range(2)]
    ref = reference(q, K, V, lens, new, table, mask="causal")
    refw = reference(q, K, V, lens, new, table, mask="window", window=90, sink=3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    first = None
    for _ in range(3):
        attn_paged_prefill_fwd(qv, cache, n, tab, seq_offsets=o, out=ov, workspace=ws[0][:need], stream=streams[0])
        ow, lw = attn_paged_prefill_fwd(qv, cache, n, tab, seq_offsets=o, mask="window", window=90, sink=3,
                                        workspace=ws[1][:need], stream=streams[1])
        torch.cuda.synchronize()
        sync_status()
        if first is None:
            first = ov.clone(), ow.clone()
        assert torch.equal(ov, first[0]) and torch.equal(ow, first[1])
    check(ov, None, ref, fmt, d)
    check(ow, lw, refw, fmt, d)
    assert (room[Hq] == 7).all() and (room[:, :, d:] == 7).all()
    assert all((w[need:] == 0xA5).all() for w in ws)
    # captured once, replayed over other lengths
    out, lse = torch.zeros((T, Hq, d), device=DEV, dtype=torch.bfloat16), torch.zeros((T, Hq), device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_paged_prefill_fwd(qv, cache, n, tab, seq_offsets=o, out=out, lse=lse, workspace=ws[0][:need])
    g.replay()
    sync_status()
    check(out, lse, ref, fmt, d)
    l2, n2 = [900, 280, 0], [61, 280, 0]
    n.copy_(dev(l2, torch.int32))
    o.copy_(dev([0, 61, 341, 341], torch.int32))
    g.replay()
    sync_status()
    check(out, lse, reference(q, K, V, l2, n2, table, mask="causal"), fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_a_pool_past_32_bits(fmt):
    """Pages whose first element lies past 2^31 (elements, and bytes)."""
    Hq, Hkv, d, page = 4, 2, 128, 256
    pages = 2 ** 31 // (Hkv * page * (d if fmt == "bf16" else d // 2)) + 40
    small, K, V = pool(fmt, 6, Hkv, page, d, seed=11)
    parts = []
    for t in small:
        if t is None:
            parts.append(None)
            continue
        big = torch.empty((pages, *t.shape[1:]), device=DEV, dtype=t.dtype)
        big[-6:] = t.to(DEV)
        parts.append(big)
    past, new = [300, 0], [100, 500]
    lens = [400, 500]
    table = table_for(lens, page, 6, seed=2)
    q = (synth.randn_bf16((600, Hq, d), synth.generator(4)).float() * 0.2).bfloat16()
    out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts), dev(lens, torch.int32),
                                      dev(np.where(table < 0, -1, table + pages - 6).astype(np.int32)),
                                      seq_offsets=dev([0, 100, 600], torch.int32))
    sync_status()
    rows = [0, 99, 100, 300, 599]
    for r in rows:
        b, i = (0, r) if r < 100 else (1, r - 100)
        n = lens[b] - new[b] + i + 1
        ref = oracle.paged_attention(q[r:r + 1].transpose(0, 1)[None], K, V, [n], np.maximum(table[b:b + 1], 0))
        check(out[r:r + 1], lse[r:r + 1], [np.swapaxes(x[0], 0, 1) for x in ref], fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_tile_that_never_comes_times_out_and_the_next_call_is_right(fmt, d):
    """The debug switch leaves block 0's K tile out: the waits on it run out
    after 20 ms, the call reports it, nothing stays behind."""
    from flashattention_attn_fwd_gb300._lib import FL_DEBUG_SKIP_KV_LOAD
    past, new = [40000, 5], [300, 20]
    parts, scales, K, V, table, q, lens, off = setup(fmt, 4, 2, d, 32, past, new, seed=12)
    args = q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table)
    ref = reference(q[-20:], K, V, lens[1:], new[1:], table[1:], mask="causal")
    for skip in (0, 5):
        attn_paged_prefill_fwd(*args, seq_offsets=dev(off), debug_flags=FL_DEBUG_SKIP_KV_LOAD, debug_arg=skip, wait_limit_ms=20)
        with pytest.raises(FlattnError) as e:
            sync_status()
        assert e.value.status == 5
        out, lse = attn_paged_prefill_fwd(*args, seq_offsets=dev(off))
        sync_status()
        check(out[-20:], lse[-20:], ref, fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_chunks_tables_append_decode_and_read_together(fmt):
    """A long prompt as it is served: tables of a stretched context, three chunks
    appended and attended (another sequence decoding beside), single tokens, the
    cache read back; against the forward over what the cache holds, and over the
    training path's rotation."""
    from flashattention_attn_fwd_gb300 import PagedKVCache, kv_append, kv_read, rope_fwd, rope_tables
    Hq, Hkv, d, page, L = 8, 2, 128, 32, 700
    cos, sin = rope_tables(4096, d, scaling="by_parts", factor=4.0, original=1024, amplitude=1.1)
    x = (synth.randn_bf16((2, L + 8, Hq + 2 * Hkv, d), synth.generator(13)).float() * 0.5).bfloat16().to(DEV)
    cache = PagedKVCache.allocate(64, page, Hkv, d, format=fmt, **(dict(k_scale=0.5, v_scale=0.25) if fmt == "e2m1" else {}))
    table = dev(table_for([L + 8, L + 8], page, 64, seed=1))
    kv_len = torch.zeros(2, dtype=torch.int32, device=DEV)
    got = [[], []]
    # (tokens of sequence 0, of sequence 1) a step
    at = [0, 0]
    for new in ((256, 1), (1, 300), (300, 0), (143, 398), (0, 1), (1, 1)):
        rows = torch.cat([x[b, at[b]:at[b] + new[b]] for b in range(2)])
        off = dev([0, new[0], sum(new)], torch.int32)
        kv_len += dev(new, torch.int32)
        q = kv_append(cache, rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], kv_len, table, seq_offsets=off, rope_cos=cos,
                      rope_sin=sin, q=rows[:, :Hq])
        out, lse = attn_paged_prefill_fwd(q, cache, kv_len, table, seq_offsets=off)
        if new == (1, 1):  # decode gives the same rows
            o2, l2 = attn_paged_decode_fwd(q[:, :, None], cache, kv_len, table)
            sync_status()
            assert (o2[:, :, 0].float() - out.float()).abs().max() <= 2.0 ** -6 * out.float().abs().max()
            assert (l2[:, :, 0] - lse).abs().max() < 1e-4
        for b in range(2):
            got[b].append(out[(0, new[0])[b]:(new[0], sum(new))[b]])
            at[b] += new[b]
    sync_status()
    assert at == [701, 701]
    off = dev([0, 701, 1402], torch.int32)
    k, v = kv_read(cache, kv_len, table, 1402, seq_offsets=off)
    qr, kr = rope_fwd(x[:, :701, :Hq].transpose(1, 2), x[:, :701, Hq:Hq + Hkv].transpose(1, 2), cos, sin)
    kc = k.view(2, 701, Hkv, d).transpose(1, 2)
    if fmt == "bf16":
        assert torch.equal(kc, kr)
    full, _ = attn_fwd(qr, kc.contiguous(), v.view(2, 701, Hkv, d).transpose(1, 2).contiguous(), mask="causal")
    sync_status()
    for b in range(2):
        diff = torch.cat(got[b]).float() - full[b].transpose(0, 1).float()
        assert diff.abs().max() <= 2e-2 and diff.norm() <= 1e-2 * full[b].float().norm()


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow_from_tile_to_tile(fmt, d):
    """Keys whose scores rise by small and by large steps (up to hundreds, past
    what a 32-bit exponential takes) in either half of a tile, for some rows and
    not for others, and fall again: the running reference has to follow."""
    Hq, Hkv, page, n = 2, 1, 64, 1500
    lens, new = [n], [130]
    pages = -(-n // page)
    parts, K, V = pool(fmt, pages, Hkv, page, d, seed=21)
    table = table_for(lens, page, pages, seed=22)
    rng = np.random.default_rng(23)
    level = np.zeros(n)
    for at, to in ((40, 1.0), (100, 3.0), (130, 9.0), (250, 2.0), (300, 20.0), (460, 21.0), (600, 60.0), (1000, 5.0),
                   (1100, 61.0), (1215, 300.0), (1300, 0.0)):
        level[at:] = to
    # every row's score of key j is about level[j] times the row's factor
    factor = np.where(np.arange(130)[:, None] % 3 == 0, 0.0, 1.0) * np.array([1.0, -0.5])[None]
    u = np.ones(d)
    q = torch.from_numpy(factor[..., None] * u * np.sqrt(d) / 8 + 0.02 * rng.normal(size=(130, Hq, d))).bfloat16()
    parts = [t.clone() if t is not None else None for t in parts]
    for j in range(n):
        pg, at = table[0, j // page], j % page
        row = level[j] * 8.0 / d * u + 0.05 * rng.normal(size=d)
        if fmt == "bf16":
            parts[0][pg, 0, at] = torch.from_numpy(row).bfloat16()
        else:
            c, s8 = oracle.quantise(row, 1.0)
            parts[0][pg, 0, at] = torch.from_numpy((c[0::2] | (c[1::2] << 4)).astype(np.uint8))
            parts[2][pg, 0, at] = torch.from_numpy(s8.astype(np.uint8))
    if fmt == "bf16":
        K = parts[0].double().numpy()
    else:
        b = parts[0].numpy()
        K = oracle.dequantise(np.stack((b & 15, b >> 4), -1).reshape(pages, Hkv, page, d), parts[2].numpy(), 1.0)
    for kw in (dict(mask="causal"), dict(mask="window", window=400, sink=110)):
        ref = reference(q, K, V, lens, new, table, **kw)
        out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts), dev(lens, torch.int32), dev(table),
                                          seq_offsets=dev([0, 130], torch.int32), **kw)
        sync_status()
        check(out, lse, ref, fmt, d)
