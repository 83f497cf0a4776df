"""A call that failed leaves nothing behind: the next one on the thread reports
its own errors alone."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import (_lib, FlattnError, PagedKVCache, attn_bwd, attn_fwd, attn_paged_decode_fwd, kv_append,
                                           sync_status, synth)
from flashattention_attn_fwd_gb300.api import _stream_ptr, _variant_desc

DEV = "cuda"


@pytest.mark.gpu
def test_calls_after_one_that_failed():
    """Waiting for a stream while it is captured is an error of the runtime (and
    ends the capture); calls after it run."""
    q, k, v = (t.to(DEV) for t in synth.attn_inputs(1, 2, 2, 200, 64, seed=1))
    kw = dict(mask="window", window=64, sink=4)
    out, lse = attn_fwd(q, k, v, **kw)
    cache = PagedKVCache.allocate(4, 16, 2, 64)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    n = torch.tensor([1], dtype=torch.int32, device=DEV)
    row = k[0, :, :1].transpose(0, 1).contiguous()
    new = q[:, :, :1].contiguous()

    def noalloc_status():
        desc = _variant_desc(1, 2, 2, 200, 200, 64, 64, stream=_stream_ptr(None))
        _lib.check(_lib.lib().fl_attn_fwd_noalloc(0, 0, 0, 0, 0, desc), "fl_attn_fwd_noalloc")
    noalloc_status()   # its set-up comes before any capture
    calls = [lambda: attn_fwd(q, k, v, **kw), lambda: attn_bwd(q, k, v, out, out, lse, **kw),
             lambda: kv_append(cache, row, row, n, table), lambda: attn_paged_decode_fwd(new, cache, n, table)]
    for call in calls:
        call()
    sync_status()
    for ask, call in [(sync_status, c) for c in calls] + [(noalloc_status, c) for c in calls]:
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(Exception):
            with torch.cuda.graph(graph):
                with pytest.raises(FlattnError) as e:
                    ask()
                assert e.value.status == 4
        call()
        sync_status()
