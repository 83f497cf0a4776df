"""Reading the cache back into tensors that the call allocates: rows that it leaves out
are zeros, written on the call's stream."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import kv_read, sync_status
from tests._left import dirty, reported
from tests._paged import pool, table_for
from tests.test_gpu_paged import DEV, dev, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_read_allocates_zeroed_rows_on_the_calls_stream(fmt):
    """Rows at negative positions, of a bad page and behind the last sequence."""
    Hkv, d, page, T = 3, 64, 16, 60
    lens, rows = [40, 5], [40, 12]
    parts, _, _ = pool(fmt, 4, Hkv, page, d, seed=8)
    cache = make_cache(parts)
    t = table_for(lens, page, 4, seed=9)
    n, off = dev(lens, torch.int32), dev([0, 40, 52], torch.int32)
    kept = [torch.full((T, Hkv, d), 7.0, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    kv_read(cache, n, dev(t), T, seq_offsets=off, k_out=kept[0], v_out=kept[1])
    sync_status()
    left = torch.zeros(T, dtype=torch.bool)
    left[40:47] = left[52:] = True
    assert all((x[left] == 7).all() and torch.isfinite(x).all() for x in kept)
    t2 = t.copy()
    t2[0, 1] = 10 ** 6
    left[16:32] = True
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s, under in ((None, None), (side, side), (side.cuda_stream, side), (0, torch.cuda.default_stream())):
        dirty(((T, Hkv, d), torch.bfloat16), stream=under)
        got = kv_read(cache, n, dev(t2), T, seq_offsets=off, stream=s)
        torch.cuda.synchronize()
        reported()
        for x, w in zip(got, kept):
            assert (x[left] == 0).all() and torch.equal(x[~left], w[~left])
