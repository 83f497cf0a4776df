"""Shared by the tests of rows that a call leaves out (test infrastructure)."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import FlattnError, sync_status
from tests.test_gpu_paged import DEV


def dirty(*shapes, stream=None):
    """Leaves NaNs in the memory that the next tensors of these sizes get."""
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
        held = [torch.full(s, float("nan"), device=DEV, dtype=t) for s, t in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del held


def reported():
    with pytest.raises(FlattnError) as e:
        sync_status()
    assert e.value.status == 6
