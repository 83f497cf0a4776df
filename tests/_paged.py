"""Builders shared by the paged-cache tests (test infrastructure)."""
import numpy as np
import torch

import oracle


def table_for(lens, page, pages, seed=0, width=None):
    """Pages for the lengths in random order, int32 [B, width] (-1 unused)."""
    rng = np.random.default_rng(seed)
    perm = rng.permutation(pages)
    need = [-(-n // page) for n in lens]
    assert sum(need) <= pages
    width = max(need + [1]) if width is None else width
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t


def pool(fmt, pages, Hkv, page, d, seed=0, k_scale=1.0, v_scale=1.0):
    """(device tensors k, v, k_scales, v_scales; fp64 values K, V)."""
    rng = np.random.default_rng(seed)
    if fmt == "bf16":
        k = torch.from_numpy(rng.normal(size=(pages, Hkv, page, d))).bfloat16()
        v = torch.from_numpy(rng.normal(size=(pages, Hkv, page, d))).bfloat16()
        return (k, v, None, None), k.double().numpy(), v.double().numpy()
    code = rng.integers(0, 16, size=(2, pages, Hkv, page, d)).astype(np.uint8)
    s8 = rng.integers(0x18, 0x38, size=(2, pages, Hkv, page, d // 16)).astype(np.uint8)
    s8[rng.random(s8.shape) < 0.02] = 0x7e  # some blocks at the largest scale,
    s8[rng.random(s8.shape) < 0.02] = 0x01  # some at the smallest,
    s8[rng.random(s8.shape) < 0.02] = 0x00  # some zero
    K, V = oracle.dequantise(code[0], s8[0], k_scale), oracle.dequantise(code[1], s8[1], v_scale)
    b = torch.from_numpy(code[..., 0::2] | (code[..., 1::2] << 4))
    return (b[0].clone(), b[1].clone(), torch.from_numpy(s8[0].copy()),
            torch.from_numpy(s8[1].swapaxes(-1, -2).copy())), K, V


def unpack(cache):
    """fp32 values (k, v) [pages, Hkv, page, d] that a cache's pages hold, and
    its codes and scales (4-bit: k codes, v codes, k scales, v scales)."""
    if cache.format == "bf16":
        return cache.k.float().cpu().numpy(), cache.v.float().cpu().numpy(), None
    def codes(x):
        x = x.cpu().numpy()
        return np.stack((x & 15, x >> 4), -1).reshape(*x.shape[:-1], -1)
    kc, vc = codes(cache.k), codes(cache.v)
    ks, vs = cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy().swapaxes(-1, -2)
    return oracle.dequantise(kc, ks, cache.k_scale), oracle.dequantise(vc, vs, cache.v_scale), (kc, vc, ks, vs)


def rope_tables(positions, rot, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(rot // 2) * 2.0 / rot)[None]
    return torch.from_numpy(np.cos(a)).float(), torch.from_numpy(np.sin(a)).float()
