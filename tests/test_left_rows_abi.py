"""What the descriptors say about rows that a call leaves out: values that are taken
and refused, before any CUDA call (no GPU)."""
import pytest

from flashattention_attn_fwd_gb300 import _lib
from tests.test_more_abi import L, no_gpu, rope_desc, turn  # noqa: F401
from tests.test_paged_abi import INV


@pytest.mark.parametrize("call", ["fl_rope_fwd", "fl_rope_bwd"])
@pytest.mark.parametrize("layout", [0x12, 0x22, 0x32, 0x40, 0x41, 0x100, -1, -0x10])
def test_rope_refuses_other_flags(L, layout, call):  # noqa: F811
    assert turn(L, rope_desc(rope_interleaved=layout), call=call) == INV


@no_gpu
@pytest.mark.parametrize("layout", [0x10, 0x11, 0x20, 0x21, 0x30, 0x31])
def test_rope_takes_its_flags(L, layout):  # noqa: F811
    for call in ("fl_rope_fwd", "fl_rope_bwd"):
        assert turn(L, rope_desc(rope_interleaved=layout), call=call) == _lib.FL_ERR_CUDA
