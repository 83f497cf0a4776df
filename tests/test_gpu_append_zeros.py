"""Zeros of both signs in a 4-bit cache: the code of -0 is -0 (e2m1(u / s) keeps
the sign), as is that of a negative value that rounds to zero."""
import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import PagedKVCache, kv_append, sync_status
from tests._paged import rope_tables, unpack

DEV = "cuda"


def _rows(d):
    """[T, 1, d] bf16: zeros of both signs among ordinary values, beside tiny
    ones, alone in their block, and in blocks whose scale is 0."""
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.normal(size=(40, 1, d))).bfloat16()
    x[:, :, 0::3] = -0.0
    x[:, :, 1::5] = 0.0
    x[1, :, ::2] = -0.01                      # rounds to -0 beside ordinary values
    x[2] = -0.0
    x[3] = 0.0
    x[4, :, :16] = torch.tensor([-0.0, 0.0] * 8)
    x[5, :, 16:32] = torch.tensor([-1e-30, 1e-30, -0.0, 0.0] * 4)   # a block whose scale is 0
    x[6] = torch.from_numpy(np.where(rng.random((1, d)) < 0.5, -448.0 * 6, -0.0)).bfloat16()
    return x


def test_the_oracle_keeps_the_sign_of_zero():
    code, s8 = oracle.quantise(np.array([[-0.0, 0.0, 1.0, -1.0] + [-0.0] * 12]), 1.0, np.float32)
    assert s8[0, 0] > 0 and list(code[0, :4]) == [8, 0, 7, 15] and (code[0, 4:] == 8).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1e30])
@pytest.mark.parametrize("rot", ["none", "half", "pairs"])
def test_append_keeps_the_sign_of_zero(d, scale, rot):
    x = _rows(d)
    T, page = x.shape[0], 16
    cache = PagedKVCache.allocate(3, page, 1, d, format="e2m1", k_scale=scale, v_scale=scale)
    table = torch.arange(3, dtype=torch.int32, device=DEV)[None]
    kw = {}
    k = x.float().numpy()
    if rot != "none":
        cos, sin = rope_tables(T, d)
        sin[::2] = 0.0                          # and a rotation that leaves zeros zero
        cos[::2] = 1.0
        kw = dict(rope_cos=cos.to(DEV), rope_sin=sin.to(DEV), rope_interleaved=rot == "pairs")
        k = oracle.rotate(x, cos.numpy(), sin.numpy(), rot == "pairs", np.float32)
    ko, vo = (torch.empty((T, 1, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kv_append(cache, x.to(DEV), x.to(DEV), torch.tensor([T], dtype=torch.int32, device=DEV), table,
              seq_offsets=torch.tensor([0, T], dtype=torch.int32, device=DEV), k_out=ko, v_out=vo, **kw)
    sync_status()
    _, _, (kc, vc, ks, vs) = unpack(cache)
    for rows, code, s8, out in ((k, kc, ks, ko), (x.float().numpy(), vc, vs, vo)):
        want, want8 = oracle.quantise(rows, np.float32(scale), np.float32)
        code = code.swapaxes(1, 2).reshape(-1, 1, d)[:T]
        assert np.array_equal(s8.swapaxes(1, 2).reshape(-1, 1, d // 16)[:T], want8)
        assert np.array_equal(code, want)
        # the values that come back carry the codes' signs too
        assert np.array_equal(np.signbit(out.float().cpu().numpy()), code >= 8)
