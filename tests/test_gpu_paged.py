"""GPU tests of the paged cache: append against the oracle's 32-bit steps
(bit for bit) and 64-bit definition, decode against the 64-bit oracle with
bounds derived per element.

Decode bound.  out = sum_j P_j v_j.  Each weight carries the score's error ds
(relative) and the rounding of P for the tensor core, half a step of its type
(bf16 2^-8, fp16 2^-11), so the sum is off by at most (2 ds + rP) sum_j P_j
|v_j| (numerator and denominator), and the result is rounded to bf16: 2^-8
|out|.  ds: d products summed in fp32, each step rounding 2^-24 of at most mag =
max_j sum_c |q_c k_c| scale, and four 32-bit steps after it (scale, maximum,
exponent): (d + 8) 2^-24 mag, plus 2^-21 for the exponential and logarithm.  A
4-bit cache's query is in fp16 after scaling by a power of two: channels below
2^-14 of the largest lose at most 2^-25 of it, 2^-25 top in all, top = max|q|
max_j sum_c |k_c| scale.  A weight too small for P's type is lost: with
the largest weight at 1 (fp16: at 2^7 or more) that is 2^-126 in bf16 (the
exponential flushes subnormals) and 2^-32 in fp16 (half of its smallest step,
2^-25, over 2^7), of every |v_j|; the sum of weights is at least the largest.
"""
import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import (FlattnError, PagedKVCache, attn_fwd, attn_paged_decode_fwd,
                                           attn_paged_decode_workspace_size, kv_append, sync_status, synth)
from tests._paged import pool, rope_tables, table_for, unpack

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dtype=None):
    x = torch.as_tensor(x)
    return (x if dtype is None else x.to(dtype)).to(DEV)


def make_cache(parts, **kw):
    return PagedKVCache(*(None if t is None else t.to(DEV) for t in parts), **kw)


def check_decode(out, lse, ref, fmt, q):
    ro, rl, amp, tot, mag, top = ref
    d = q.shape[-1]
    ds = ((d + 8) * 2.0 ** -24 * mag + 2.0 ** -21)[..., None]
    if fmt == "e2m1":
        ds = ds + 2.0 ** -25 * top[..., None]
    rp = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -11
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    lost = 2.0 ** -126 if fmt == "bf16" else 2.0 ** -32
    # 2 % for the products of two errors
    tol = 1.02 * ((2 * ds + rp) * amp + 2.0 ** -8 * np.abs(ro) + lost * tot)
    err = np.abs(got - ro)
    assert (err <= tol).all(), float((err / tol).max())
    if lse is not None:
        gl = lse.double().cpu().numpy()
        live = np.isfinite(rl)
        assert np.array_equal(live, np.isfinite(gl)) and (gl[~live] == -np.inf).all()
        assert (np.abs(gl[live] - rl[live]) <= (2 * ds[..., 0] + 2.0 ** -20)[live] + 2.0 ** -22 * np.abs(rl[live])).all()


DECODE = [
    # fmt, B, Hq, Hkv, Lq, d, page, lens, kwargs
    ("e2m1", 1, 1, 1, 1, 64, 16, [1], {}),
    ("e2m1", 3, 8, 2, 1, 64, 16, [15, 16, 17], {}),
    ("e2m1", 4, 8, 2, 1, 128, 32, [0, 31, 33, 400], {}),
    ("e2m1", 2, 4, 4, 1, 128, 256, [255, 513], {}),
    ("e2m1", 2, 12, 4, 3, 64, 64, [200, 2], dict(mask="causal")),
    ("e2m1", 2, 8, 1, 2, 128, 128, [130, 700], dict(mask="causal")),
    ("e2m1", 1, 32, 1, 2, 128, 16, [333], dict(mask="causal")),
    ("e2m1", 1, 40, 1, 1, 64, 64, [100], {}),
    ("e2m1", 2, 4, 2, 1, 128, 16, [900, 40], dict(mask="window", window=100, sink=4)),
    ("e2m1", 2, 6, 2, 4, 64, 32, [777, 3], dict(mask="window", window=33, sink=17)),
    ("e2m1", 2, 4, 2, 1, 64, 16, [300, 200], dict(mask="window", window=1, sink=0)),
    ("e2m1", 2, 4, 2, 2, 64, 16, [300, 60], dict(mask="window", window=50, sink=200)),
    ("e2m1", 2, 4, 2, 1, 64, 16, [300, 60], dict(mask="window", window=1 << 30, sink=0)),
    ("e2m1", 2, 8, 2, 1, 64, 32, [500, 90], dict(score_mod="softcap", softcap=5.0)),
    ("e2m1", 2, 8, 2, 2, 128, 32, [500, 90], dict(mask="causal", score_mod="alibi")),
    ("bf16", 1, 1, 1, 1, 64, 16, [1], {}),
    ("bf16", 3, 8, 2, 1, 128, 16, [0, 16, 129], {}),
    ("bf16", 2, 12, 4, 3, 64, 64, [200, 2], dict(mask="causal")),
    ("bf16", 1, 64, 2, 2, 128, 128, [333], dict(mask="causal")),
    ("bf16", 2, 16, 1, 1, 128, 256, [300, 257], {}),
    ("bf16", 2, 6, 2, 4, 128, 32, [777, 3], dict(mask="window", window=33, sink=17)),
    ("bf16", 2, 8, 2, 1, 64, 32, [500, 90], dict(score_mod="softcap", softcap=5.0, scale=0.3)),
    ("bf16", 2, 8, 2, 2, 64, 16, [500, 90], dict(mask="window", window=64, sink=1, score_mod="alibi")),
]


# a table this wide (with missing pages) lets a sequence grow past what a
# cluster of CTAs takes: the call then cuts all units' tiles as one line
WIDE = 9000


@pytest.mark.parametrize("wide", [False, True], ids=["cluster", "line"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x) for x in c[:7]) + "-" + str(c[7][-1]) + "-" +
                         "-".join(f"{a}{b}" for a, b in c[8].items()))
def test_decode_against_the_oracle(case, wide):
    fmt, B, Hq, Hkv, Lq, d, page, lens, kw = case
    pages = sum(-(-n // page) for n in lens) + 3
    parts, K, V = pool(fmt, pages, Hkv, page, d, seed=d + page, k_scale=0.75 if fmt == "e2m1" else 1.0,
                       v_scale=1.5 if fmt == "e2m1" else 1.0)
    cache = make_cache(parts, k_scale=0.75, v_scale=1.5) if fmt == "e2m1" else make_cache(parts)
    table = table_for(lens, page, pages, seed=1, width=-(-WIDE // page) if wide else None)
    g = synth.generator(len(lens) + Hq)
    q = synth.randn_bf16((B, Hq, Lq, d), g)
    if fmt == "e2m1":
        q = (q.float() * 0.2).bfloat16()  # scales reach 448: scores of ordinary size
    okw, gkw = dict(kw), dict(kw)
    if kw.get("score_mod") == "alibi":
        s = synth.alibi_slopes(Hq)
        okw["slopes"], gkw["alibi_slopes"] = s.numpy(), s.to(DEV)
    ref = oracle.paged_attention(q, K, V, lens, np.maximum(table, 0), **okw)
    out, lse = attn_paged_decode_fwd(q.to(DEV), cache, dev(lens, torch.int32), dev(table), **gkw)
    sync_status()
    check_decode(out, lse, ref, fmt, q)


@pytest.mark.parametrize("wide", [False, True], ids=["cluster", "line"])
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_decode_many_pieces_and_row_blocks(fmt, wide):
    """Long ragged lengths: units shared by several CTAs, CTAs with several
    units, and M = 64 rows in two row blocks."""
    lens = [4000, 1, 0, 2777, 16, 900, 3333]
    page, Hkv, d = 16, 2, 64
    pages = sum(-(-n // page) for n in lens) + 1
    parts, K, V = pool(fmt, pages, Hkv, page, d, seed=4)
    table = table_for(lens, page, pages, seed=2, width=-(-WIDE // page) if wide else None)
    cache = make_cache(parts)
    for G, Lq in ((4, 1), (32, 2)):
        q = (synth.randn_bf16((len(lens), Hkv * G, Lq, d), synth.generator(3)).float() * 0.2).bfloat16()
        ref = oracle.paged_attention(q, K, V, lens, np.maximum(table, 0), mask="causal") \
            if G == 4 else None
        out, lse = attn_paged_decode_fwd(q.to(DEV), cache, dev(lens, torch.int32), dev(table), mask="causal")
        sync_status()
        if G == 4:
            check_decode(out, lse, ref, fmt, q)
        else:
            for h in (0, 31, 32, 63):  # heads of both row blocks of both key heads
                ref = oracle.paged_attention(q[:, h:h + 1], K[:, h // G:h // G + 1], V[:, h // G:h // G + 1], lens,
                                             np.maximum(table, 0), mask="causal")
                check_decode(out[:, h:h + 1], lse[:, h:h + 1], ref, fmt, q[:, h:h + 1])


@pytest.mark.parametrize("wide", [False, True], ids=["cluster", "line"])
def test_decode_more_sequences_than_threads(wide):
    """B = 300 (the plan scans several chunks), lengths 0 to 70."""
    B, page, Hkv, d = 300, 16, 1, 64
    lens = [(7 * b) % 71 for b in range(B)]
    pages = sum(-(-n // page) for n in lens) + 1
    parts, K, V = pool("bf16", pages, Hkv, page, d, seed=5)
    table = table_for(lens, page, pages, seed=3, width=-(-WIDE // page) if wide else None)
    q = synth.randn_bf16((B, 4, 1, d), synth.generator(9))
    out, lse = attn_paged_decode_fwd(q.to(DEV), make_cache(parts), dev(lens, torch.int32), dev(table))
    sync_status()
    check_decode(out, lse, oracle.paged_attention(q, K, V, lens, np.maximum(table, 0)), "bf16", q)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_decode_long_window_cut_as_a_line(fmt):
    """A window and sinks of more keys than a cluster takes, over stale pages
    (NaNs) before and between them, several sequences."""
    B, Hq, Hkv, Lq, d, page = 2, 4, 1, 2, 64, 32
    W, S = 9000, 70
    lens, kw = [9400, 300], dict(mask="window", window=W, sink=S)
    pages = sum(-(-n // page) for n in lens) + 2
    parts, K, V = pool(fmt, pages, Hkv, page, d, seed=13)
    table = table_for(lens, page, pages, seed=12)
    q = (synth.randn_bf16((B, Hq, Lq, d), synth.generator(14)).float() * 0.2).bfloat16()
    ref = oracle.paged_attention(q, K, V, lens, np.maximum(table, 0), **kw)
    parts = [t.clone() if t is not None else None for t in parts]
    for j in range(S, lens[0] - Lq - W + 1):  # keys that no row of sequence 0 sees
        pg, at = table[0, j // page], j % page
        if fmt == "bf16":
            parts[0][pg, :, at] = float("nan")
            parts[1][pg, :, at] = float("nan")
        else:
            parts[2][pg, :, at] = 0x7f
            parts[3][pg, :, :, at] = 0x7f
    t2 = table.copy()
    t2[0, 4:12] = -7
    out, lse = attn_paged_decode_fwd(q.to(DEV), make_cache(parts), dev(lens, torch.int32), dev(t2), **kw)
    sync_status()
    check_decode(out, lse, ref, fmt, q)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_decode_ignores_what_no_row_sees(fmt):
    """Stale NaNs behind the last token, between sinks and window, in other
    pages and in missing pages (-1 or out of range) change nothing."""
    B, Hq, Hkv, Lq, d, page = 2, 4, 2, 2, 64, 16
    lens, kw = [123, 250], dict(mask="window", window=40, sink=5)
    parts, K, V = pool(fmt, 32, Hkv, page, d, seed=6)
    table = table_for(lens, page, 32, seed=4)
    q = (synth.randn_bf16((B, Hq, Lq, d), synth.generator(1)).float() * 0.2).bfloat16()
    ref = oracle.paged_attention(q, K, V, lens, np.maximum(table, 0), **kw)
    parts = [t.clone() if t is not None else None for t in parts]
    for b, n in enumerate(lens):
        seen = set(range(5)) | set(range(n - Lq - 40 + 1, n))
        for j in range(-(-n // page) * page):
            if j in seen:
                continue
            pg, at = table[b, j // page], j % page
            if fmt == "bf16":
                parts[0][pg, :, at] = float("nan")
                parts[1][pg, :, at] = float("inf")
            else:
                parts[2][pg, :, at] = 0x7f      # e4m3 NaN
                parts[3][pg, :, :, at] = 0xff
    t2 = table.copy()
    t2[0, 1:4] = -1                              # no key of pages 1 .. 3 is seen
    t2[1, 1:12] = 10 ** 6
    out, lse = attn_paged_decode_fwd(q.to(DEV), make_cache(parts), dev(lens, torch.int32), dev(t2), **kw)
    sync_status()
    check_decode(out, lse, ref, fmt, q)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("wide", [False, True], ids=["cluster", "line"])
def test_decode_reports_a_bad_page_and_recovers(fmt, wide):
    lens, page = [100, 64], 16
    parts, K, V = pool(fmt, 16, 2, page, 64, seed=7)
    table = table_for(lens, page, 16, seed=5, width=WIDE // page if wide else None)
    q = (synth.randn_bf16((2, 4, 1, 64), synth.generator(2)).float() * 0.2).bfloat16()
    cache = make_cache(parts)
    for bad in (-1, 16, 2 ** 31 - 1, -2 ** 31):
        t2 = table.copy()
        t2[0, 2] = bad
        out, lse = attn_paged_decode_fwd(q.to(DEV), cache, dev(lens, torch.int32), dev(t2))
        with pytest.raises(FlattnError) as e:
            sync_status()
        assert e.value.status == 6
        # the page's keys are left out, the other sequence is untouched
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    out, lse = attn_paged_decode_fwd(q.to(DEV), cache, dev(lens, torch.int32), dev(table))
    sync_status()
    check_decode(out, lse, oracle.paged_attention(q, K, V, lens, np.maximum(table, 0)), fmt, q)


def test_decode_lengths_past_the_table_are_clamped():
    parts, K, V = pool("bf16", 8, 1, 16, 64, seed=8)
    table = np.array([[3, 1], [5, 0]], np.int32)
    q = synth.randn_bf16((2, 2, 1, 64), synth.generator(3))
    out, lse = attn_paged_decode_fwd(q.to(DEV), make_cache(parts), dev([10 ** 9, -5], torch.int32), dev(table))
    sync_status()
    check_decode(out, lse, oracle.paged_attention(q, K, V, [32, 0], table), "bf16", q)
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("wide", [False, True], ids=["cluster", "line"])
def test_decode_strides_streams_workspace_and_repeatability(fmt, wide):
    """Token-major q and out, a table with padded rows, a given workspace with
    a guard, another stream; the same call gives the same bits."""
    B, Hq, Hkv, Lq, d, page = 3, 8, 2, 2, 128, 32
    lens = [1000, 37, 513]
    parts, K, V = pool(fmt, 64, Hkv, page, d, seed=9)
    table = table_for(lens, page, 64, seed=6, width=WIDE // page + 1 if wide else None)
    wide = np.full((B, table.shape[1] + 5), 10 ** 7, np.int32)
    wide[:, :table.shape[1]] = table
    tq = (synth.randn_bf16((B, Lq, Hq, d), synth.generator(4)).float() * 0.2).bfloat16()
    q = tq.to(DEV).transpose(1, 2)
    cache = make_cache(parts)
    dt = dev(wide)[:, :table.shape[1]]
    n = attn_paged_decode_workspace_size(q, cache, dt)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    outs = []
    s = torch.cuda.Stream()
    kv = dev(lens, torch.int32)
    torch.cuda.synchronize()
    for i in range(3):
        buf = torch.full((B, Lq + 1, Hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        out, lse = attn_paged_decode_fwd(q, cache, kv, dt, mask="causal", out=buf[:, :Lq].transpose(1, 2),
                                         workspace=ws[:n], stream=s if i else None)
        torch.cuda.synchronize()
        assert (buf[:, Lq] == 7.0).all()
        outs.append((out.clone(), lse.clone()))
    sync_status()
    assert (ws[n:] == 0xA5).all()
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
    check_decode(outs[0][0], outs[0][1], oracle.paged_attention(q.cpu(), K, V, lens, np.maximum(table, 0), mask="causal"),
                 fmt, q)
    with pytest.raises(FlattnError):
        attn_paged_decode_fwd(q, cache, kv, dt, workspace=ws[:n - 16])
    with pytest.raises(ValueError):
        attn_paged_decode_fwd(q[..., ::2], cache, kv, dt)


def test_decode_extreme_queries_4bit():
    """Rows of very large, very small and zero queries, and one with a wide
    range of channels: the fp16 scaling is per row."""
    lens = [200]
    parts, K, V = pool("e2m1", 16, 1, 16, 128, seed=10)
    table = table_for(lens, 16, 16, seed=7)
    q = synth.randn_bf16((1, 8, 1, 128), synth.generator(5)).float()
    q[0, 1] *= 1e30
    q[0, 2] *= 1e-30
    q[0, 3] = 0.0
    q[0, 4, 0, 1:] *= 1e-4
    q[0, 5] *= 3e-39     # subnormal in bf16
    q = q.bfloat16()
    scale = torch.tensor([0.02, 0.02e-30, 1.0, 1.0, 0.02, 1.0, 0.02, 0.02])
    for h in range(8):
        sc = float(scale[h])
        out, lse = attn_paged_decode_fwd(q[:, h:h + 1].contiguous().to(DEV), make_cache(parts), dev(lens, torch.int32),
                                         dev(table), scale=sc)
        sync_status()
        check_decode(out, lse, oracle.paged_attention(q[:, h:h + 1], K, V, lens, np.maximum(table, 0), scale=sc),
                     "e2m1", q[:, h:h + 1])


def test_decode_pool_beyond_32_bit_offsets():
    """A pool of more than 2^32 elements (and bytes): the last pages."""
    Hkv, page, d = 8, 256, 128
    pages = (1 << 32) // (Hkv * page * d) + 8
    k = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    k[-2:] = torch.randn(k[-2:].shape, generator=g, device=DEV).bfloat16()
    v[-2:] = torch.randn(v[-2:].shape, generator=g, device=DEV).bfloat16()
    q = synth.randn_bf16((1, 16, 1, d), synth.generator(6))
    table = np.array([[pages - 1, pages - 2]], np.int32)
    cache = PagedKVCache(k, v)
    out, lse = attn_paged_decode_fwd(q.to(DEV), cache, dev([400], torch.int32), dev(table))
    sync_status()
    ref = oracle.paged_attention(q, k[-2:].cpu(), v[-2:].cpu(), [400], np.array([[1, 0]]))
    check_decode(out, lse, ref, "bf16", q)
    new = synth.randn_bf16((1, Hkv, d), synth.generator(7)).to(DEV)
    kv_append(cache, new, new, dev([401], torch.int32), dev(table))
    sync_status()
    assert torch.equal(k[pages - 2, :, 400 % page], new[0]) and torch.equal(v[pages - 2, :, 400 % page], new[0])


# ------------------------------------------------------------------- append

APPEND = [
    # fmt, B, new tokens, past tokens, Hq, Hkv, d, page, rot, interleaved, values
    ("bf16", 1, [1], [0], 1, 1, 64, 16, 64, False, False),
    ("e2m1", 1, [1], [0], 1, 1, 64, 16, 64, False, True),
    ("e2m1", 3, [1, 1, 1], [15, 16, 300], 8, 2, 128, 16, 128, False, True),
    ("bf16", 3, [5, 0, 40], [3, 9, 31], 6, 2, 128, 32, 64, False, True),
    ("e2m1", 4, [0, 17, 1, 33], [2, 0, 64, 7], 12, 4, 64, 64, 32, True, True),
    ("e2m1", 2, [129, 70], [1, 250], 7, 7, 128, 256, 128, True, False),
    ("bf16", 2, [129, 70], [0, 250], 0, 3, 64, 128, 16, True, True),
    ("e2m1", 2, [20, 3], [5, 6], 8, 8, 64, 32, 0, False, True),
    ("bf16", 2, [20, 3], [5, 6], 4, 1, 128, 16, 96, False, False),
    ("e2m1", 40, [3] * 40, [2] * 40, 4, 2, 128, 16, 96, False, True),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[:2] + c[4:]))
def test_append_against_the_oracle(case):
    fmt, B, new, past, Hq, Hkv, d, page, rot, inter, values = case
    total = [n + m for n, m in zip(new, past)]
    pages = sum(-(-n // page) for n in total) + 3
    parts, _, _ = pool(fmt, pages, Hkv, page, d, seed=11)
    ksc, vsc = (0.8, 1.7) if fmt == "e2m1" else (1.0, 1.0)
    cache = make_cache(parts, k_scale=ksc, v_scale=vsc)
    before = unpack(cache)
    table = table_for(total, page, pages, seed=8, width=max(-(-n // page) for n in total) + 2)
    T, pad = sum(new), 3
    rng = np.random.default_rng(12)
    # one fused projection, rows of it padded: strided views
    x = rng.normal(size=(T + pad, Hq + 2 * Hkv + 1, d))
    x[:, ::3, 7] *= 30.0
    x[:, 1::3, 16:32] *= 1e-4
    x = torch.from_numpy(x).bfloat16()
    if T > 3:
        x[3, Hq, :16] = 0.0
    xd = x.to(DEV)
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:Hq + 2 * Hkv]
    cos, sin = rope_tables(max(total) + 2, rot) if rot else (None, None)
    off = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    kw = {}
    if rot:
        kw.update(rope_cos=cos.to(DEV), rope_sin=sin.to(DEV), rope_interleaved=inter)
    if Hq:
        kw.update(q=q, q_out=torch.full((T + pad, Hq, d), 9.0, dtype=torch.bfloat16, device=DEV))
    if values:
        kw.update(k_out=torch.full((T + pad, Hkv, d), 9.0, dtype=torch.bfloat16, device=DEV),
                  v_out=torch.full((T + pad, Hkv, d), 9.0, dtype=torch.bfloat16, device=DEV))
    r = kv_append(cache, k, v, dev(total, torch.int32), dev(table), seq_offsets=dev(off), **kw)
    sync_status()
    assert r is kw.get("q_out")
    pos = np.concatenate([np.arange(m, m + n) for n, m in zip(new, past)]).astype(int)
    seq = np.repeat(np.arange(B), new)
    where, at = table[seq, pos // page], pos % page

    def turned(t, dtype):
        t = t[:T].cpu().double().numpy()
        return oracle.rotate(t, cos.numpy()[pos], sin.numpy()[pos], inter, dtype) if rot else t.astype(dtype)
    rows = {"k": turned(k, np.float32), "v": v[:T].cpu().float().numpy()}
    if Hq:
        want = torch.from_numpy(turned(q, np.float32)).bfloat16()
        assert torch.equal(r[:T].cpu(), want)
        assert (r[T:] == 9.0).all()
        exact = turned(q, np.float64)
        # one rounding to bf16 of a value with three 32-bit roundings
        assert (np.abs(r[:T].cpu().double().numpy() - exact) <= 2.0 ** -8 * np.abs(exact) * (1 + 2.0 ** -8) +
                3 * 2.0 ** -24 * np.abs(x[:T, :Hq].double().numpy()).max(-1, keepdims=True) * 2).all()
    after = unpack(cache)
    held = {}
    if fmt == "bf16":
        held = {n: torch.from_numpy(t).bfloat16().float().numpy() for n, t in rows.items()}
        for i, n in enumerate("kv"):
            assert np.array_equal(after[i][where, :, at], held[n])
    else:
        for i, (n, sc) in enumerate((("k", ksc), ("v", vsc))):
            code, s8 = oracle.quantise(rows[n], sc, np.float32)
            assert np.array_equal(after[2][2 + i][where, :, at], s8), n
            assert np.array_equal(after[2][i][where, :, at], code), n
            held[n] = oracle.dequantise(code, s8, sc)
            # the 64-bit definition: half of the widest step times the scale,
            # a border case included
            exact = turned(k, np.float64) if n == "k" else v[:T].cpu().double().numpy()
            s = np.repeat(oracle.paged.e4m3_values()[s8] * sc, 16, -1)
            assert (np.abs(held[n] - exact) <= s * 1.001 + 2.0 ** -10 * sc * 6).all()
    if values:
        for n in "kv":
            got = kw[n + "_out"]
            assert torch.equal(got[:T].cpu(), torch.from_numpy(held[n].astype(np.float32)).bfloat16()), n
            assert (got[T:] == 9.0).all()
    # nothing else in the pool changed
    mask = np.ones(after[0].shape[:1] + after[0].shape[2:3], bool)
    mask[where, at] = False
    for i in range(2):
        assert np.array_equal(after[i].swapaxes(1, 2)[mask], before[i].swapaxes(1, 2)[mask])


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_append_in_place_and_without_offsets(fmt):
    """q_out = q, k_out = k, v_out = v; one token per sequence, some of which
    take no part (kv_len 0) and stay untouched."""
    B, Hq, Hkv, d, page = 5, 4, 2, 64, 16
    cache = PagedKVCache.allocate(16, page, Hkv, d, format=fmt)
    lens = [3, 0, 16, 17, 0]
    table = table_for(lens, page, 16, seed=9)
    g = synth.generator(10)
    q, k, v = (synth.randn_bf16((B, H, d), g) for H in (Hq, Hkv, Hkv))
    cos, sin = rope_tables(32, d)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    kv_append(cache, kd, vd, dev(lens, torch.int32), dev(table), rope_cos=cos.to(DEV), rope_sin=sin.to(DEV), q=qd,
              q_out=qd, k_out=kd, v_out=vd)
    sync_status()
    K, V, _ = unpack(cache)
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.equal(qd[b].cpu(), q[b]) and torch.equal(kd[b].cpu(), k[b]) and torch.equal(vd[b].cpu(), v[b])
            continue
        p = np.array([n - 1])
        want = oracle.rotate(q[b:b + 1], cos.numpy()[p], sin.numpy()[p], False, np.float32)
        assert torch.equal(qd[b].cpu(), torch.from_numpy(want[0]).bfloat16())
        pg, at = table[b, (n - 1) // page], (n - 1) % page
        assert np.array_equal(kd[b].float().cpu().numpy(), K[pg, :, at].astype(np.float32))
        assert np.array_equal(vd[b].float().cpu().numpy(), V[pg, :, at].astype(np.float32))


def test_append_reports_what_is_out_of_range_and_leaves_it():
    Hkv, d, page = 1, 64, 16
    cos, sin = rope_tables(40, d)
    cos, sin = cos.to(DEV), sin.to(DEV)
    k = torch.ones((1, Hkv, d), dtype=torch.bfloat16, device=DEV)
    for lens, table in (([33], [[0, 1]]),            # past the table's columns
                        ([20], [[0, -1]]), ([20], [[0, 4]]), ([20], [[0, 2 ** 31 - 1]]),   # no such page
                        ([41], [[0, 1, 2]])):        # no rotation for position 40
        cache = PagedKVCache.allocate(4, page, Hkv, d)
        q = k.clone()
        kv_append(cache, k, k, dev(lens, torch.int32), dev(table, torch.int32), rope_cos=cos, rope_sin=sin, q=q, q_out=q)
        with pytest.raises(FlattnError) as e:
            sync_status()
        assert e.value.status == 6
        assert (cache.k == 0).all() and (cache.v == 0).all() and torch.equal(q, k)
    # positions before the first token are no error
    cache = PagedKVCache.allocate(4, page, Hkv, d)
    kv_append(cache, k, k, dev([-7], torch.int32), dev([[9]], torch.int32))
    sync_status()
    assert (cache.k == 0).all()


@pytest.mark.parametrize("scale", [1.0, 0.7, 3.3e-5, 4096.0])
def test_append_rounding_borders_of_every_scale(scale):
    """For every e4m3 scale s, blocks whose largest magnitude fixes it (6 s) and
    whose other values sit on a border of the 4-bit codes, or one bf16 step to
    either side: the codes are those of the correctly rounded quotient."""
    e4 = oracle.paged.e4m3_values()[1:]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    blocks = []
    for s in e4:
        m = torch.from_numpy(mids * s * scale).bfloat16()
        bits = m.view(torch.int16)
        up, dn = (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)
        top = torch.tensor([6 * s * scale]).bfloat16()
        for v in (torch.cat((top, m, -m, m[:1])), torch.cat((top, up, -dn, up[:1])), torch.cat((-top, -up, dn, dn[:1]))):
            blocks.append(v)
    rng = np.random.default_rng(3)
    blocks += [torch.from_numpy(rng.normal(size=16) * 10.0 ** rng.uniform(-8, 6)).bfloat16() for _ in range(2000)]
    x = torch.stack(blocks)
    x = torch.cat((x, torch.zeros(-len(x) % 8, 16, dtype=torch.bfloat16))).reshape(-1, 1, 128)  # [T, 1, 128]
    T, page = x.shape[0], 256
    pages = -(-T // page)
    cache = PagedKVCache.allocate(pages, page, 1, 128, format="e2m1", k_scale=scale, v_scale=scale)
    table = np.arange(pages, dtype=np.int32)[None]
    kv_append(cache, x.to(DEV), x.to(DEV), dev([T], torch.int32), dev(table), seq_offsets=dev([0, T], torch.int32))
    sync_status()
    with np.errstate(over="ignore"):
        code, s8 = oracle.quantise(x.float().numpy(), np.float32(scale), np.float32)
    _, _, (kc, vc, ks, vs) = unpack(cache)
    for got_c, got_s in ((kc, ks), (vc, vs)):
        got_c, got_s = got_c.reshape(-1, 1, 128)[:T], got_s.reshape(-1, 1, 8)[:T]
        assert np.array_equal(got_s, s8) and np.array_equal(got_c, code)


def test_append_infinities_saturate_their_block():
    cache = PagedKVCache.allocate(2, 16, 1, 64, format="e2m1")
    k = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    k[0, 0, 3], k[0, 0, 20] = float("inf"), -float("inf")
    kv_append(cache, k, k, dev([1], torch.int32), dev([[1]], torch.int32))
    sync_status()
    K, _, _ = unpack(cache)
    row = K[1, 0, 0]
    assert row[3] == 448 * 6 and row[20] == -448 * 6 and (np.delete(row[:32], [3, 20]) == 0).all()
    # 1 / 6 is 10.67 sixty-fourths: scale 11 / 64, 1 over it rounds to code 6
    assert (row[32:] == 6 * 11 / 64).all()


# ------------------------------------------------- the operators as one run

@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_prompt_append_and_decode_steps_as_a_model_runs_them(fmt):
    """A prompt through window attention with sinks, its keys and values
    appended, then tokens generated one at a time: each step's decode equals
    full attention over the tokens so far (oracle, on the stored values)."""
    Hq, Hkv, d, page, W, S = 4, 2, 64, 16, 24, 3
    L0, steps = 53, 14
    cache = PagedKVCache.allocate(12, page, Hkv, d, format=fmt, **({} if fmt == "bf16" else dict(k_scale=0.05, v_scale=0.05)))
    table = dev(table_for([L0 + steps], page, 12, seed=10))
    cos, sin = rope_tables(L0 + steps, d)
    cos, sin = cos.to(DEV), sin.to(DEV)
    g = synth.generator(11)
    x = synth.randn_bf16((L0 + steps, Hq + 2 * Hkv, d), g).to(DEV)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    ko, vo = (torch.empty((L0 + steps, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    off = dev([0, L0], torch.int32)
    qr = kv_append(cache, k[:L0], v[:L0], dev([L0], torch.int32), table, seq_offsets=off, rope_cos=cos, rope_sin=sin,
                   q=q[:L0], k_out=ko[:L0], v_out=vo[:L0])
    out, _ = attn_fwd(qr.transpose(0, 1)[None], ko[:L0].transpose(0, 1)[None], vo[:L0].transpose(0, 1)[None],
                      mask="window", window=W, sink=S)
    sync_status()
    ro, _ = oracle.attention(qr.transpose(0, 1)[None].cpu(), ko[:L0].transpose(0, 1)[None].cpu(),
                             vo[:L0].transpose(0, 1)[None].cpu(), mask="window", window=W, sink=S)
    assert np.abs(out.double().cpu().numpy() - ro).max() <= 2e-2
    for t in range(L0, L0 + steps):
        n = dev([t + 1], torch.int32)
        qt = kv_append(cache, k[t:t + 1], v[t:t + 1], n, table, rope_cos=cos, rope_sin=sin, q=q[t:t + 1],
                       k_out=ko[t:t + 1], v_out=vo[t:t + 1])
        o, l = attn_paged_decode_fwd(qt.unsqueeze(2), cache, n, table, mask="window", window=W, sink=S)
        sync_status()
        K, V, _ = unpack(cache)
        ref = oracle.paged_attention(qt.unsqueeze(2).cpu(), K, V, [t + 1], table.cpu().numpy(), mask="window", window=W,
                                     sink=S)
        check_decode(o, l, ref, fmt, qt.unsqueeze(2))
        # the cache holds what k_out and v_out say
        r2, _ = oracle.attention(qt.unsqueeze(2).cpu(), ko[:t + 1].transpose(0, 1)[None].cpu().double()[:, :, list(range(S)) + list(range(t + 1 - W, t + 1))],
                                 vo[:t + 1].transpose(0, 1)[None].cpu().double()[:, :, list(range(S)) + list(range(t + 1 - W, t + 1))])
        assert np.abs(o.double().cpu().numpy() - r2).max() <= 2e-2


def test_captured_step_replays_and_graphs_with_own_workspaces_overlap():
    """append + decode captured in two graphs (own workspaces), replayed with
    new inputs and lengths written in place, also at the same time on two
    streams."""
    Hq, Hkv, d, page, B = 8, 2, 64, 16, 3
    cos, sin = rope_tables(600, d)
    cos, sin = cos.to(DEV), sin.to(DEV)
    sync_status()  # the library's first call, before any capture

    class Step:
        def __init__(self, seed):
            self.cache = PagedKVCache.allocate(120, page, Hkv, d, format="e2m1", k_scale=0.05, v_scale=0.05)
            g = synth.generator(seed)
            self.table = dev(table_for([590] * B, page, 120, seed=seed))
            self.x = synth.randn_bf16((B, Hq + 2 * Hkv, d), g).to(DEV)
            self.kv = dev([1, 1, 1], torch.int32)
            q = torch.empty((B, Hq, 1, d), dtype=torch.bfloat16, device=DEV)
            self.qo = torch.empty((B, Hq, d), dtype=torch.bfloat16, device=DEV)
            self.ws = torch.empty(attn_paged_decode_workspace_size(q, self.cache, self.table), dtype=torch.uint8, device=DEV)
            self.out, self.lse = torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV)
            self.run()
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.run()

        def run(self):
            kv_append(self.cache, self.x[:, Hq:Hq + Hkv], self.x[:, Hq + Hkv:], self.kv, self.table, rope_cos=cos,
                      rope_sin=sin, q=self.x[:, :Hq], q_out=self.qo)
            attn_paged_decode_fwd(self.qo.unsqueeze(2), self.cache, self.kv, self.table, mask="causal", out=self.out,
                                  lse=self.lse, workspace=self.ws)
    steps = [Step(1), Step(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n in (1, 2, 17, 300, 301):
        for i, s in enumerate(steps):
            s.kv.copy_(torch.tensor([n, n + 250, max(n - 5, 0)], dtype=torch.int32))
            s.x.copy_(synth.randn_bf16(tuple(s.x.shape), synth.generator(100 * n + i)))
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.graph.replay()
        torch.cuda.synchronize()
        sync_status()
        for s in steps:
            K, V, _ = unpack(s.cache)
            ref = oracle.paged_attention(s.qo.unsqueeze(2).cpu(), K, V, s.kv.cpu().numpy(), s.table.cpu().numpy(), mask="causal")
            check_decode(s.out, s.lse, ref, "e2m1", s.qo.unsqueeze(2))


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("wide", [False, True], ids=["cluster", "line"])
def test_decode_sequences_that_share_pages(fmt, wide):
    """Pages may be read through several rows of the table, and twice through one
    row: the same queries over the same pages give the same result, and a page
    named twice counts twice."""
    page, n = 16, 100
    parts, K, V = pool(fmt, 8, 2, page, 64, seed=31)
    row = [3, 5, 3, 1, 0, 3, 7]
    width = WIDE // page if wide else len(row)
    table = np.zeros((3, width), np.int32)
    table[:, :len(row)] = row
    lens = [n, n, 37]
    q = (synth.randn_bf16((1, 4, 1, 64), synth.generator(8)).float() * 0.3).bfloat16().expand(3, 4, 1, 64).contiguous()
    out, lse = attn_paged_decode_fwd(q.to(DEV), make_cache(parts), dev(lens, torch.int32), dev(table))
    sync_status()
    check_decode(out, lse, oracle.paged_attention(q, K, V, lens, table), fmt, q)
    if not wide:
        assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])
