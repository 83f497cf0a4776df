"""The chunk attention's waits that may give up: in a warp that goes on as a whole
(elect.sync, __syncwarp, shuffles) the lanes take one answer.  A lane that saw the
limit pass while another saw the tile arrive would leave the warp for good, and the
next elect.sync of the others would wait for it without an end."""
import os
import re

import pytest
import torch

from tests.test_gpu_paged import DEV, dev, make_cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_wait_that_may_give_up_is_voted_on():
    """No GPU: each call of pf_wait in the kernel stands in a vote of the warp, and no
    lone test of a barrier decides a branch."""
    txt = open(os.path.join(ROOT, "flashattention_attn_fwd_gb300", "csrc", "paged_prefill.cuh")).read()
    body = txt[txt.index("paged_prefill_kernel("):]
    calls = [m.start() for m in re.finditer(r"\bpf_wait\(", body)]
    assert calls
    for at in calls:
        assert body[:at].rstrip().endswith("__all_sync(0xffffffffu,"), body[at - 60:at + 60]
    # probes: their results meet in a vote
    names = re.findall(r"(\w+) = ptx::mbar_test_wait\(", body)
    votes = " ".join(re.findall(r"__all_sync\(0xffffffffu, ([^;{]*)", body))
    assert names and all(re.search(rf"\b{n}\b", votes) for n in names)
    for n in names:
        uses = [m.start() for m in re.finditer(rf"\b{n}\b(?! =)", body)]
        assert len(uses) == 1, n  # in the vote alone


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("past,new", [([5000, 3], [300, 20]), ([0, 700], [257, 1]), ([9000], [5])], ids=str)
def test_waits_that_run_out_at_any_tile_end_the_call(fmt, d, past, new):
    """Whichever key tile of block 0 is left out, the call ends within a few of its
    limits, says so if a wait ran out, and the next one is right to the bit."""
    from flashattention_attn_fwd_gb300 import FlattnError, attn_paged_prefill_fwd, sync_status
    from flashattention_attn_fwd_gb300._lib import FL_DEBUG_SKIP_KV_LOAD
    from tests.test_gpu_prefill import setup
    parts, scales, K, V, table, q, lens, off = setup(fmt, 4, 2, d, 32, past, new, seed=41)
    args = q.to(DEV), make_cache(parts, **scales), dev(lens, torch.int32), dev(table)
    want, lse = attn_paged_prefill_fwd(*args, seq_offsets=dev(off))
    sync_status()
    ran_out = 0
    for skip in range(10):
        attn_paged_prefill_fwd(*args, seq_offsets=dev(off), debug_flags=FL_DEBUG_SKIP_KV_LOAD, debug_arg=skip, wait_limit_ms=2)
        try:
            sync_status()
        except FlattnError as e:
            assert e.status == 5
            ran_out += 1
        got, l2 = attn_paged_prefill_fwd(*args, seq_offsets=dev(off))
        sync_status()
        assert torch.equal(got, want) and torch.equal(l2, lse)
    assert ran_out
