"""Chunk attention, rows behind the last sequence: left as they are in tensors that the
call is given; zeros, with a log-sum-exp of -inf, in those that it allocates."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import attn_paged_prefill_fwd, sync_status, synth
from tests._left import dirty
from tests._paged import pool, table_for
from tests.test_gpu_paged import DEV, dev, make_cache

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("T,new", [(9, [2, 3]), (700, [130, 0, 5]), (64, [0, 0]), (40, [40]), (5000, [1])], ids=str)
def test_chunk_rows_behind_the_last_sequence(fmt, T, new):
    Hq, Hkv, d, page = 6, 2, 64, 16
    past = [40 + 3 * b for b in range(len(new))]
    lens = [p + n for p, n in zip(past, new)]
    pages = sum(-(-n // page) for n in lens)
    parts, _, _ = pool(fmt, pages, Hkv, page, d, seed=5)
    cache, table = make_cache(parts), dev(table_for(lens, page, pages, seed=6))
    q = (synth.randn_bf16((T, Hq, d), synth.generator(7)).float() * 0.2).bfloat16().to(DEV)
    n, total = dev(lens, torch.int32), sum(new)
    off = dev([0] + [sum(new[:b + 1]) for b in range(len(new))], torch.int32)
    kept, kl = torch.full((T, Hq, d), 7.0, device=DEV, dtype=torch.bfloat16), torch.full((T, Hq), 7.0, device=DEV)
    attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off, out=kept, lse=kl)
    sync_status()
    assert (kept[total:] == 7).all() and (kl[total:] == 7).all()
    shapes = ((T, Hq, d), torch.bfloat16), ((T, Hq), torch.float32)

    def whole(out, lse):
        assert torch.equal(out[:total], kept[:total]) and (out[total:] == 0).all()
        assert torch.equal(lse[:total], kl[:total]) and (lse[total:] == -INF).all()
    dirty(*shapes)
    whole(*attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off))
    # one given, one allocated
    dirty(*shapes)
    out, lse = attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off, out=torch.full_like(kept, 7.0))
    assert torch.equal(out, kept) and (lse[total:] == -INF).all()
    dirty(*shapes)
    out, lse = attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off, lse=torch.full_like(kl, 7.0))
    assert torch.equal(lse, kl) and (out[total:] == 0).all()
    dirty(*shapes)
    out, lse = attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off, return_lse=False)
    assert lse is None and (out[total:] == 0).all()
    # another stream, by object and by handle
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        dirty(*shapes, stream=side)
        got = attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off, stream=s)
        side.synchronize()
        whole(*got)
    # captured with all rows in use, replayed with fewer
    off2 = off.clone()
    off2[-1] = T
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off2)
    off2.copy_(off)
    got[0].fill_(float("nan"))
    got[1].fill_(float("nan"))
    graph.replay()
    sync_status()
    whole(*got)
