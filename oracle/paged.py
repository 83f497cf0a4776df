"""CPU oracle for the paged key/value cache: rotation of new tokens, the 4-bit
format and attention over pages (test infrastructure; the same import rules
as the rest of ``oracle``).

Rotation and attention are the definitions in 64 bits.  ``quantise`` takes a
dtype: in float64 it is the definition, in float32 the stated sequence of
rounded 32-bit steps that decides values on a rounding border.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64, softmax_rows

__all__ = ["rotate", "quantise", "dequantise", "paged_attention"]

# magnitudes of the low three bits of an e2m1 code
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    """The 127 finite non-negative e4m3 values by code (bias 7, subnormals)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def _nearest(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest grid value (ascending) to each x >= 0, ties to
    the even index, saturating.  Exact: midpoints are representable."""
    x = x.astype(np.float64)
    mid = (grid[1:] + grid[:-1]) / 2.0
    lo = np.searchsorted(mid, x, side="left")    # a tie goes down ...
    hi = np.searchsorted(mid, x, side="right")   # ... or up
    return np.where(lo % 2 == 0, lo, hi)


def rotate(x, cos, sin, interleaved: bool, dtype=np.float64) -> np.ndarray:
    """x [T, H, d] rotated by cos, sin [T, rot / 2] in `dtype`, every product
    and sum rounded to it."""
    x = _f64(x).astype(dtype)
    c, s = _f64(cos).astype(dtype)[:, None], _f64(sin).astype(dtype)[:, None]
    half = c.shape[-1]
    y = x.copy()
    ia, ib = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def quantise(x, scale: float, dtype=np.float64):
    """Codes [.., d] (4 bits each) and e4m3 block-scale codes [.., d / 16] of
    x / scale: block scale max|u| / 6, codes u / s, rounded to nearest even."""
    x = np.asarray(x, dtype=dtype)
    u = (x * (dtype(1) / dtype(scale))).reshape(*x.shape[:-1], -1, 16)
    s8 = _nearest(np.abs(u).max(-1) * (dtype(1) / dtype(6)), e4m3_values())
    s = e4m3_values()[s8].astype(dtype)[..., None]
    t = np.where(s > 0, u / np.where(s > 0, s, 1), dtype(0))
    code = _nearest(np.abs(t), E2M1) | np.where(np.signbit(t), 8, 0)
    return code.reshape(x.shape), s8


def dequantise(code, s8, scale: float) -> np.ndarray:
    """The values of codes [.., d] with block scales [.., d / 16]."""
    code = np.asarray(code)
    val = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = e4m3_values()[np.asarray(s8)]
    return (val.reshape(*code.shape[:-1], -1, 16) * s[..., None]).reshape(code.shape) * float(np.float32(scale))


def paged_attention(q, keys, values, kv_len, table, *, mask: str = "none", window: int = 0, sink: int = 0,
                    score_mod: str = "none", slopes=None, softcap: float | None = None, scale: float | None = None):
    """Attention of q [B, Hq, Lq, d] over pools keys, values [pages, Hkv,
    page, d] through table [B, n].  Returns (out, lse) and what error
    bounds are made of: amp = sum_j P_j |v_j| and tot = sum_j |v_j| over the
    visible keys per output value; mag = max_j sum_c |q_c k_c| scale and top =
    max|q_c| max_j sum_c |k_c| scale per row."""
    q, keys, values = _f64(q), _f64(keys), _f64(values)
    B, Hq, Lq, d = q.shape
    Hkv, page = keys.shape[1:3]
    scale = 1.0 / np.sqrt(d) if scale is None else float(scale)
    out, amp, tot = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, mag, top = np.full((B, Hq, Lq), -np.inf), np.zeros((B, Hq, Lq)), np.zeros((B, Hq, Lq))
    for b in range(B):
        n = min(max(int(kv_len[b]), 0), table.shape[1] * page)
        j = np.arange(n)
        for h in range(Hq):
            for i in range(Lq):
                p = n - Lq + i
                vis = np.ones(n, bool) if mask == "none" else j <= p
                if mask == "window":
                    vis &= (j > p - window) | (j < sink)
                jj = j[vis]
                if jj.size == 0:
                    continue
                pg = np.asarray(table)[b][jj // page]
                k, v = keys[pg, h // (Hq // Hkv), jj % page], values[pg, h // (Hq // Hkv), jj % page]
                t = scale * (k @ q[b, h, i])
                mag[b, h, i] = scale * (np.abs(k) @ np.abs(q[b, h, i])).max()
                top[b, h, i] = scale * np.abs(q[b, h, i]).max() * np.abs(k).sum(1).max()
                if score_mod == "softcap":
                    t = softcap * np.tanh(t / softcap)
                if score_mod == "alibi":
                    t = t + float(slopes[h]) * (jj - p)
                    mag[b, h, i] += np.abs(float(slopes[h]) * (jj - p)).max()
                P, l = softmax_rows(t[None])
                out[b, h, i], lse[b, h, i] = P[0] @ v, l[0]
                amp[b, h, i] = P[0] @ np.abs(v)
                tot[b, h, i] = np.abs(v).sum(0)
    return out, lse, amp, tot, mag, top
