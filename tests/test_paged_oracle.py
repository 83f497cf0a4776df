"""Pins of the paged-cache oracle (CPU): the number formats against torch's
e4m3 and hand-written tables, rotation against complex multiplication, paged
attention against the decode oracle on the gathered cache."""
import numpy as np
import pytest
import torch

import oracle
from oracle.paged import E2M1, _nearest, e4m3_values


def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())
    x = torch.rand(20000, generator=torch.Generator().manual_seed(0)) * torch.logspace(-4, 2.6, 20000)
    want = x.clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(_nearest(x.numpy(), e4m3_values()), want)


@pytest.mark.parametrize("x,code", [(0.0, 0), (0.25, 0), (0.26, 1), (0.74, 1), (0.75, 2), (1.25, 2), (1.26, 3),
                                    (1.75, 4), (2.5, 4), (2.51, 5), (3.5, 6), (5.0, 6), (5.01, 7), (9.0, 7)])
def test_e2m1_rounding_table(x, code):
    assert _nearest(np.array([x]), E2M1)[0] == code


def test_quantise_round_trip_bounds_and_special_blocks():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(40, 64)) * np.exp(rng.normal(size=(40, 1)))
    x[3] = 0.0
    x[4, :16] = 1e-7          # scale rounds to zero: stored as zeros
    code, s8 = oracle.quantise(x, 0.5)
    y = oracle.dequantise(code, s8, 0.5)
    s = np.repeat(e4m3_values()[s8] * 0.5, 16, axis=-1)
    # half of the widest step (4 to 6) times the scale; up to 6 / 16 more where
    # the scale was rounded down and the largest magnitude saturates
    assert (np.abs(x - y) <= s * 1.0 + 1e-6).all()
    assert (y[3] == 0).all() and (y[4, :16] == 0).all()
    # what is stored is stored again unchanged
    code2, s82 = oracle.quantise(y, 0.5)
    live = s8 > 0
    assert np.array_equal(s82[live & (np.abs(y.reshape(40, 4, 16)).max(-1) == 6 * e4m3_values()[s8] * 0.5)],
                          s8[live & (np.abs(y.reshape(40, 4, 16)).max(-1) == 6 * e4m3_values()[s8] * 0.5)])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(2)
    x, a = rng.normal(size=(5, 3, 64)), rng.normal(size=(5, 16))
    y = oracle.rotate(x, np.cos(a), np.sin(a), interleaved)
    ia, ib = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * a)[:, None]
    assert np.allclose(y[..., ia], z.real, atol=1e-13) and np.allclose(y[..., ib], z.imag, atol=1e-13)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    back = oracle.rotate(y, np.cos(a), -np.sin(a), interleaved)
    assert np.allclose(back, x, atol=1e-12)


def test_paged_attention_is_decode_attention_on_the_gathered_cache():
    rng = np.random.default_rng(3)
    B, Hq, Hkv, Lq, d, page, n = 3, 4, 2, 2, 8, 4, 5
    q = rng.normal(size=(B, Hq, Lq, d))
    pool_k, pool_v = rng.normal(size=(20, Hkv, page, d)), rng.normal(size=(20, Hkv, page, d))
    table = rng.permutation(20)[:B * n].reshape(B, n)
    kv_len = np.array([20, 7, 2])
    k = pool_k[table].transpose(0, 2, 1, 3, 4).reshape(B, Hkv, n * page, d)
    v = pool_v[table].transpose(0, 2, 1, 3, 4).reshape(B, Hkv, n * page, d)
    for mask in ("none", "causal"):
        o, l, *_ = oracle.paged_attention(q, pool_k, pool_v, kv_len, table, mask=mask)
        ro, rl = oracle.decode_attention(q, k, v, kv_len, causal=mask == "causal")
        assert np.allclose(o, ro, atol=1e-13) and np.allclose(l, rl, atol=1e-13)
    # a window that covers everything is causal; sinks join a small window
    o, l, *_ = oracle.paged_attention(q, pool_k, pool_v, kv_len, table, mask="window", window=99)
    assert np.allclose(o, oracle.decode_attention(q, k, v, kv_len, causal=True)[0], atol=1e-13)
    o, *_ = oracle.paged_attention(q, pool_k, pool_v, kv_len, table, mask="window", window=1, sink=1)
    t = np.stack([k[0, 0, 0] @ q[0, 0, 1], k[0, 0, 19] @ q[0, 0, 1]]) / np.sqrt(d)
    w = np.exp(t - t.max())
    assert np.allclose(o[0, 0, 1], (w[0] * v[0, 0, 0] + w[1] * v[0, 0, 19]) / w.sum(), atol=1e-13)


def test_sink_visibility_counts():
    vis = oracle.visibility("window", 20, 20, window=4, sink=3)
    assert vis.sum(1).tolist() == [1, 2, 3, 4, 5, 6] + [7] * 14
    assert np.array_equal(oracle.visibility("window", 20, 20, window=4), oracle.visibility("window", 20, 20, window=4, sink=0))
    assert np.array_equal(oracle.visibility("window", 20, 20, window=1, sink=20), oracle.visibility("causal", 20, 20))
