"""The device wait limit bounds a step of the pipeline, not a walk of the
backward over all query tiles of a key tile: walks that last several limits end
with their results."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import _lib, attn_bwd, attn_fwd, sync_status, synth
from flashattention_attn_fwd_gb300.api import _stream_ptr, _variant_desc

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_walks_longer_than_the_wait_limit(d):
    """65536 queries of 8 heads: a walk is 4096 steps of about a microsecond, the
    limit one millisecond."""
    B, Hq, Hkv, Lq, Lk, limit_ms = 1, 8, 1, 65536, 256 * 128, 1
    g = synth.generator(d)
    q, do = (synth.randn_bf16((B, Hq, Lq, d), g).to(DEV) for _ in range(2))
    k, v = (synth.randn_bf16((B, Hkv, Lk, d), g).to(DEV) for _ in range(2))
    out, lse = attn_fwd(q, k, v)
    want = attn_bwd(q, k, v, out, do, lse)
    sync_status()
    L = _lib.lib()
    desc = _variant_desc(B, Hq, Hkv, Lq, Lk, d, d, stream=_stream_ptr(None), debug=(0, -1, limit_ms))
    got = [torch.zeros_like(t) for t in (q, k, v)]
    ws = torch.empty(L.fl_attn_bwd_workspace_size(desc), dtype=torch.uint8, device=DEV)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    _lib.check(L.fl_attn_bwd(*(t.data_ptr() for t in (q, k, v, out, do, lse, *got, ws)), ws.numel(), desc), "fl_attn_bwd")
    end.record()
    sync_status()
    # 256 walks on fewer than 256 blocks at once: two in a row, each longer than the limit
    assert begin.elapsed_time(end) > 2 * limit_ms
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
