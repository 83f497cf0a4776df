"""Window with sinks, backward, under a cap far above the scores: cap tanh(s / cap)
is s to within s^3 / (3 cap^2) < 2^-20 (|s| < 20, cap 1e5), so the gradients are
those without a cap, within their bounds, however large the cap."""
import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import (attn_bwd, attn_decode_fwd, attn_fwd, attn_paged_decode_fwd, sync_status, synth)
from tests._paged import pool, table_for
from tests.test_gpu_paged import check_decode, make_cache
from tests.test_gpu_sink import _bounds, _inputs, _within

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e5, 1e9, 3e38])
@pytest.mark.parametrize("case", [
    # (B, Hq, Hkv, L, d, dv, window, sink): up to 64 tokens, few keys a row, first rows
    (2, 4, 2, 40, 64, 64, 9, 3), (1, 2, 1, 64, 128, 128, 64, 2), (1, 2, 2, 300, 64, 64, 40, 4), (1, 2, 1, 450, 32, 32, 100, 9),
    (1, 2, 2, 700, 64, 64, 300, 4), (1, 2, 2, 640, 64, 128, 200, 4), (1, 2, 1, 600, 128, 128, 100, 4),
], ids=lambda c: "-".join(str(x) for x in c))
def test_a_cap_far_above_the_scores_changes_nothing(case, softcap):
    B, Hq, Hkv, L, d, dv, window, sink = case
    q, k, v, dout = _inputs(B, Hq, Hkv, L, d, dv, seed=3 * L + d)
    a = [t.to(DEV) for t in (q, k, v, dout)]
    kw = dict(mask="window", window=window, sink=sink, score_mod="softcap", softcap=softcap)
    out, lse = attn_fwd(*a[:3], **kw)
    grads = attn_bwd(*a[:3], out, a[3], lse, **kw)
    sync_status()
    r, e = _bounds(q, k, v, dout, window, sink)
    _within(out, r["out"], e["out"], "out")
    for name, g in zip(("dq", "dk", "dv"), grads):
        _within(g, r[name], e[name], name)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e5, 3.4e38])
@pytest.mark.parametrize("fmt", ["bf16", "e2m1", "contiguous"])
def test_a_cap_far_above_the_scores_changes_no_decode(fmt, softcap):
    lens, page, Hkv, d = [100, 37], 16, 2, 64
    parts, K, V = pool("bf16" if fmt == "contiguous" else fmt, 16, Hkv, page, d, seed=3)
    table = table_for(lens, page, 16, seed=1)
    q = (synth.randn_bf16((2, 4, 1, d), synth.generator(2)).float() * 0.2).bfloat16()
    ref = oracle.paged_attention(q, K, V, lens, np.maximum(table, 0))
    kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if fmt == "contiguous":
        k, v = (t[np.maximum(table, 0)].transpose(1, 2).flatten(2, 3).contiguous().to(DEV) for t in parts[:2])
        out, lse = attn_decode_fwd(q.to(DEV), k, v, kv_len, score_mod="softcap", softcap=softcap)
    else:
        out, lse = attn_paged_decode_fwd(q.to(DEV), make_cache(parts), kv_len, torch.from_numpy(table).to(DEV),
                                         score_mod="softcap", softcap=softcap)
    sync_status()
    check_decode(out, lse, ref, "bf16" if fmt == "contiguous" else fmt, q)
