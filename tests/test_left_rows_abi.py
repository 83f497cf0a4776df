"""What the descriptors say about rows that a call leaves out: values that are taken
and refused, before any CUDA call (no GPU)."""
import pytest

from flashattention_attn_fwd_gb300 import _lib
from tests.test_more_abi import L, no_gpu, prefill, prefill_desc, rope_desc, turn  # noqa: F401
from tests.test_paged_abi import INV, cache


@pytest.mark.parametrize("call", ["fl_rope_fwd", "fl_rope_bwd"])
@pytest.mark.parametrize("layout", [0x12, 0x22, 0x32, 0x40, 0x41, 0x100, -1, -0x10])
def test_rope_refuses_other_flags(L, layout, call):  # noqa: F811
    assert turn(L, rope_desc(rope_interleaved=layout), call=call) == INV


@no_gpu
@pytest.mark.parametrize("layout", [0x10, 0x11, 0x20, 0x21, 0x30, 0x31])
def test_rope_takes_its_flags(L, layout):  # noqa: F811
    for call in ("fl_rope_fwd", "fl_rope_bwd"):
        assert turn(L, rope_desc(rope_interleaved=layout), call=call) == _lib.FL_ERR_CUDA


@pytest.mark.parametrize("fill", [4, 8, 0x10, 0x80000000])
def test_chunks_refuse_other_fills(L, fill):  # noqa: F811
    assert prefill(L, cache(), prefill_desc(fill=fill)) == INV
    assert prefill(L, cache(format=1), prefill_desc(fill=fill | 3)) == INV


@no_gpu
@pytest.mark.parametrize("fill", [0, 1, 2, 3])
def test_chunks_take_their_fills(L, fill):  # noqa: F811
    for kw in (dict(), dict(lse=0)):
        assert prefill(L, cache(), prefill_desc(fill=fill), **kw) == _lib.FL_ERR_CUDA
    assert prefill(L, cache(), prefill_desc(fill=fill, Lq=2), off=0) == _lib.FL_ERR_CUDA
