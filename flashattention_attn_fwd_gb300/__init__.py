"""GB300-native fused attention forward for attention variants.

The computation lives in the CUDA library ``libflattn.so`` (C ABI in
``include/flattn.h``); this package holds the build step, a thin ctypes
binding with the same entry-point names, the FLOP/byte accounting used for
the roofline, and the seeded synthetic-input generators.
"""
from .api import (FlattnError, attn_bwd, attn_decode_fwd, attn_fwd, attention, diffattn_bwd,  # noqa: F401
                  diff_attention, diffattn_fwd,
                  evoformer_col_gated_attn_fwd, evoformer_gated_attn_fwd, sync_status)
from .paged import (PagedKVCache, attn_paged_decode_fwd, attn_paged_decode_workspace_size,  # noqa: F401
                    attn_paged_prefill_fwd, attn_paged_prefill_workspace_size, kv_append, kv_read)
from .rotary import rope, rope_bwd, rope_fwd, rope_tables  # noqa: F401

__all__ = ["attn_fwd", "diffattn_fwd", "diffattn_bwd", "evoformer_gated_attn_fwd", "evoformer_col_gated_attn_fwd",
           "attn_decode_fwd", "PagedKVCache", "kv_append", "attn_paged_decode_fwd",
           "attn_paged_decode_workspace_size", "attn_paged_prefill_fwd", "attn_paged_prefill_workspace_size", "kv_read",
           "rope", "rope_fwd", "rope_bwd", "rope_tables", "attn_bwd", "attention", "diff_attention", "sync_status", "FlattnError"]
