"""Chunk attention under caps far above a row's scores: what other rows, other
sequences' rows and keys that nobody sees hold must not cost a row its accuracy.

Bound, beside that of tests/test_gpu_prefill.py without its cap term.  Where |t| <=
0.46 cap the scores go through a polynomial within 1e-6 of tanh, relative, in 32-bit
steps (tests/test_poly_constants.py), whose folded coefficients add 2^-22: at most
1.3e-6 |t|.  Beyond, cap (1 - 2 / (1 + e^2y)): exponential and reciprocal within 2^-22
each and a rounding of cap's size give 2^-20 cap <= 2.2 x 2^-20 |t| = 2.1e-6 |t|.  |t| is
at most mag: 2.1e-6 mag whichever way a score goes."""
import numpy as np
import pytest
import torch

from flashattention_attn_fwd_gb300 import attn_paged_prefill_fwd, sync_status
from tests.test_gpu_paged import DEV, dev, make_cache
from tests.test_gpu_prefill import check, reference, setup

pytestmark = pytest.mark.gpu


def check_any_cap(out, lse, ref, fmt, d, rows):
    part = [x[rows] for x in ref]
    part[4] = part[4] * (1.0 + 2.1e-6 * 2.0 ** 24 / (d + 8))  # into the bound's (d + 8) 2^-24 mag
    check(out[rows], lse[rows], part, fmt, d)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap", [80.0, 1e5, 1e7])
@pytest.mark.parametrize("where", ["nowhere", "another token", "the next sequence", "unseen keys"])
def test_large_scores_elsewhere_cost_a_row_nothing(fmt, d, softcap, where):
    Hq, Hkv, page = 4, 2, 64
    past, new = [300, 20], [37, 25]
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=31)
    rows = np.ones(sum(new), bool)
    if where == "another token":
        q[[3, 50]] *= 100 * softcap
        rows[[3, 50]] = False
    elif where == "the next sequence":
        q[37:] *= 100 * softcap
        rows[37:] = False
    elif where == "unseen keys" and fmt == "bf16":
        for b, n in enumerate(lens):
            at = n % page
            assert at
            parts[0][table[b, n // page], :, at:] = 1e30
    kw = dict(mask="causal", score_mod="softcap", softcap=softcap)
    ref = reference(q, K, V, lens, new, table, **kw)
    out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table),
                                      seq_offsets=dev(off), **kw)
    sync_status()
    check_any_cap(out.cpu(), lse.cpu(), ref, fmt, d, rows)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("softcap", [0.5, 20.0])
def test_rows_with_scores_on_both_sides_of_the_polynomials_range(fmt, softcap):
    Hq, Hkv, d, page = 4, 2, 64, 32
    past, new = [200, 0], [60, 140]
    parts, scales, K, V, table, q, lens, off = setup(fmt, Hq, Hkv, d, page, past, new, seed=32)
    q[::3] *= 16
    kw = dict(mask="window", window=90, sink=3, score_mod="softcap", softcap=softcap)
    ref = reference(q, K, V, lens, new, table, **kw)
    out, lse = attn_paged_prefill_fwd(q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table),
                                      seq_offsets=dev(off), **kw)
    sync_status()
    check_any_cap(out, lse, ref, fmt, d, np.arange(sum(new)))
