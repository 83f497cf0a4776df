"""GPU parity of sliding-window attention with sinks, forward and backward,
against the 64-bit oracle, with bounds derived per element.

Score error.  A score is d products summed in fp32 on the tensor core (each
step within 2^-22 of mag = max sum_c |q_c k_c| scale), transformed (softcap: the
fitted tanh, 2^-20 cap) and exponentiated against a reference or LSE in fp32
(2^-18 in all): a weight is off by a factor 1 + ds,
ds = (d + 8) 2^-22 mag + 2^-20 cap + 2^-18.
Forward.  P is rounded to bf16 (2^-8) before P V, the sum of weights carries ds
too, and the result is rounded: (2 ds + 2^-8) sum P |v| + 2^-8 |out|.
Backward.  dV = P^T dO with P in bf16: (ds + 2^-8) sum P |dO| + 2^-8 |dv|.
dS = P (dP - D) (1 - tanh^2): dP is an fp32 sum, off by eP = 2^-22 (dv + 8) sum
|dO v|; D = sum P dP is summed in fp32 from such products, off by eD = sum P
(2 ds |dP| + eP) where rows see few keys (window + sink <= 64, or L <= 512), else
it is dO . O with the forward's O, off by the forward's bound: eD = sum |dO| eO;
the difference and sech^2 (fp16 pairs, 2^-11 of 1) and dS
itself (bf16, 2^-8) are rounded:
eS = P (eD + eP) + (ds + 2^-8 + 2^-20) |dS| + 2^-11 P |dP - D| (softcap).
Query 0 sees one key: its dS is zero.
dQ and dK are scale sum eS |k|, scale sum eS |q|, rounded to bf16 (2^-8).
5 % for products of errors and fp32 sums over rows.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import (_lib, attention, attn_bwd, attn_fwd, synth, sync_status)

DEV = "cuda"
gpu = pytest.mark.gpu


def _bounds(q, k, v, dout, window, sink, score_mod="none", slopes=None, softcap=None, scale=None):
    """fp64 outputs, gradients and their error bounds, one (b, h) at a time."""
    q, k, v = (t.double().numpy() for t in (q, k, v))
    do = None if dout is None else dout.double().numpy()
    B, Hq, L, d = q.shape
    Hkv, dv = k.shape[1], v.shape[-1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    vis = oracle.visibility("window", L, L, window=window, sink=sink)
    r = {n: np.zeros(s) for n, s in (("out", (B, Hq, L, dv)), ("lse", (B, Hq, L)), ("dq", q.shape), ("dk", k.shape),
                                     ("dv", v.shape))}
    e = {n: np.zeros_like(x) for n, x in r.items()}
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = scale * (q[b, h] @ k[b, g].T)
            mag = np.where(vis, scale * (np.abs(q[b, h]) @ np.abs(k[b, g]).T), 0).max(1)
            t = oracle.apply_score_mod(s, score_mod, slope=None if slopes is None else float(slopes[h]), cap=softcap)
            if score_mod == "alibi":
                # the bias reaches the score in fp32 parts of a tile's size
                mag = mag + abs(float(slopes[h])) * L
            P, lse = oracle.attention.__globals__["softmax_rows"](np.where(vis, t, -np.inf))
            ds = ((d + 8) * 2.0 ** -22 * mag + 2.0 ** -20 * (softcap or 0.0) + 2.0 ** -18)[:, None]
            o = P @ v[b, g]
            eo = (2 * ds + 2.0 ** -8) * (P @ np.abs(v[b, g])) + 2.0 ** -8 * np.abs(o)
            r["out"][b, h], e["out"][b, h] = o, eo
            r["lse"][b, h], e["lse"][b, h] = lse, 2 * ds[:, 0]
            if do is None:
                continue
            D0 = do[b, h]
            dP = D0 @ v[b, g].T
            df = dP - (P * dP).sum(1, keepdims=True)
            sech = 1.0 - np.tanh(s / softcap) ** 2 if softcap else 1.0
            dS = P * df * sech
            dS[0] = 0.0
            eP = 2.0 ** -22 * (dv + 8) * (np.abs(D0) @ np.abs(v[b, g]).T)
            few = window + sink <= 64 or L <= 512
            eD = (P * (2 * ds * np.abs(dP) + eP)).sum(1, keepdims=True) if few else (np.abs(D0) * eo).sum(1, keepdims=True)
            eS = P * (eD + eP) + (ds + 2.0 ** -8 + 2.0 ** -20) * np.abs(dS)
            if softcap:
                eS = eS + 2.0 ** -11 * P * np.abs(df)
            eS[0] = 0.0
            r["dq"][b, h], e["dq"][b, h] = scale * dS @ k[b, g], scale * eS @ np.abs(k[b, g])
            r["dk"][b, g] += scale * dS.T @ q[b, h]
            e["dk"][b, g] += scale * eS.T @ np.abs(q[b, h])
            r["dv"][b, g] += P.T @ D0
            e["dv"][b, g] += ((ds + 2.0 ** -8) * P).T @ np.abs(D0)
    for n in ("dq", "dk", "dv"):
        e[n] = e[n] + 2.0 ** -8 * np.abs(r[n])
    return r, e


def _within(got, want, bound, name):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), name
    x = np.abs(g - want) / (1.05 * bound + 1e-30)
    assert x.max() <= 1, (name, float(x.max()))


def _inputs(B, Hq, Hkv, L, d, dv, seed):
    q, k, v = synth.attn_inputs(B, Hq, Hkv, L, d, dv, seed=seed)
    return q, k, v, synth.randn_bf16((B, Hq, L, dv), synth.generator(seed + 1))


def _mods(mod, Hq):
    if mod == "alibi":
        s = synth.alibi_slopes(Hq)
        return dict(score_mod="alibi", alibi_slopes=s.to(DEV)), dict(score_mod="alibi", slopes=s.numpy())
    if mod:
        return dict(score_mod="softcap", softcap=mod), dict(score_mod="softcap", softcap=mod)
    return {}, {}


FWD = [
    # B, Hq, Hkv, L, d, dv, window, sink, mod
    (1, 1, 1, 1, 64, 64, 1, 1, None), (1, 2, 1, 2, 32, 32, 1, 1, None), (2, 2, 2, 129, 64, 64, 1, 1, None),
    (1, 2, 2, 128, 64, 64, 5, 4, None), (1, 2, 2, 300, 64, 64, 64, 4, None), (1, 1, 1, 700, 64, 64, 128, 4, None),
    (1, 3, 1, 700, 64, 64, 200, 128, None), (1, 2, 2, 900, 64, 64, 100, 129, None), (1, 2, 2, 900, 32, 64, 129, 300, None),
    (1, 2, 2, 513, 64, 64, 64, 600, None), (1, 2, 2, 513, 64, 64, 600, 8, None), (1, 4, 2, 1000, 128, 128, 130, 17, None),
    (1, 2, 2, 1000, 128, 64, 256, 140, None), (1, 2, 2, 640, 128, 32, 33, 2, None), (1, 2, 2, 640, 64, 128, 33, 200, None),
    (1, 4, 2, 777, 64, 64, 70, 4, "alibi"), (1, 4, 2, 777, 128, 128, 70, 40, "alibi"), (1, 4, 4, 777, 64, 64, 70, 4, 5.0),
    (1, 2, 1, 777, 32, 32, 150, 256, 30.0), (3, 5, 5, 385, 64, 64, 100, 3, None),
]


@gpu
@pytest.mark.parametrize("case", FWD, ids=lambda c: "-".join(str(x) for x in c))
def test_forward(case):
    B, Hq, Hkv, L, d, dv, window, sink, mod = case
    q, k, v, _ = _inputs(B, Hq, Hkv, L, d, dv, seed=L + d)
    gkw, okw = _mods(mod, Hq)
    out, lse = attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), mask="window", window=window, sink=sink, **gkw)
    sync_status()
    r, e = _bounds(q, k, v, None, window, sink, **okw)
    _within(out, r["out"], e["out"], "out")
    _within(lse, r["lse"], e["lse"], "lse")


BWD = [
    (1, 1, 1, 1, 64, 64, 1, 1, None), (1, 2, 2, 129, 64, 64, 1, 1, None), (1, 2, 2, 301, 64, 64, 64, 4, None),
    (1, 4, 2, 700, 64, 64, 100, 4, None), (2, 2, 1, 515, 32, 32, 64, 130, None), (1, 2, 2, 902, 128, 128, 129, 4, None),
    (1, 1, 1, 2500, 64, 64, 30, 4, None), (1, 2, 1, 1500, 128, 128, 40, 300, None), (1, 2, 2, 900, 64, 128, 100, 5, None),
    (1, 4, 2, 640, 64, 64, 70, 4, "alibi"), (1, 2, 2, 641, 64, 64, 70, 140, 5.0), (1, 2, 1, 642, 128, 128, 70, 4, 30.0),
    (1, 2, 2, 400, 64, 64, 500, 7, None), (1, 2, 2, 400, 64, 64, 20, 500, None), (1, 2, 2, 643, 32, 32, 128, 128, 5.0),
]


@gpu
@pytest.mark.parametrize("case", BWD, ids=lambda c: "-".join(str(x) for x in c))
def test_backward(case):
    B, Hq, Hkv, L, d, dv, window, sink, mod = case
    q, k, v, dout = _inputs(B, Hq, Hkv, L, d, dv, seed=2 * L + d)
    gkw, okw = _mods(mod, Hq)
    qd, kd, vd, dd = (t.to(DEV) for t in (q, k, v, dout))
    kw = dict(mask="window", window=window, sink=sink, **gkw)
    out, lse = attn_fwd(qd, kd, vd, **kw)
    grads = attn_bwd(qd, kd, vd, out, dd, lse, **kw)
    sync_status()
    r, e = _bounds(q, k, v, dout, window, sink, **okw)
    for n, g in zip(("dq", "dk", "dv"), grads):
        _within(g, r[n], e[n], n)


@gpu
@pytest.mark.parametrize("L,window,sink", [(2, 1, 1), (3, 1, 1), (5, 2, 1), (40, 1, 1), (300, 2, 1), (300, 4, 4), (64, 200, 1)])
def test_gradients_of_few_keys_keep_their_precision(L, window, sink):
    """Rows that see few keys: dS cancels, and the gradients stay within what
    the two bf16 roundings (dS, then the result: 2^-8 each at most) and fp32
    allow in the 2-norm."""
    q, k, v, dout = _inputs(2, 4, 2, L, 64, 64, seed=L)
    kw = dict(mask="window", window=window, sink=sink)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    out, lse = attn_fwd(qd, kd, vd, **kw)
    grads = attn_bwd(qd, kd, vd, out, dout.to(DEV), lse, **kw)
    sync_status()
    r, e = _bounds(q, k, v, dout, window, sink)
    for n, g in zip(("dq", "dk", "dv"), grads):
        _within(g, r[n], e[n], n)
        assert np.linalg.norm(g.double().cpu().numpy() - r[n]) <= 2.0 ** -7 * np.linalg.norm(r[n]), n
    assert (grads[0][:, :, 0] == 0).all()


@gpu
def test_one_token_has_no_gradient_but_v():
    q, k, v, dout = _inputs(2, 4, 2, 1, 128, 128, seed=5)
    kw = dict(mask="window", window=3, sink=2)
    out, lse = attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), **kw)
    dq, dk, dv = attn_bwd(q.to(DEV), k.to(DEV), v.to(DEV), out, dout.to(DEV), lse, **kw)
    sync_status()
    assert (dq == 0).all() and (dk == 0).all()
    assert torch.equal(out.cpu(), v.repeat_interleave(2, 1))
    want = dout.double().reshape(2, 2, 2, 1, 128).sum(2).numpy()
    assert (np.abs(dv.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20).all()


@gpu
def test_gradients_against_differences_and_through_autograd():
    """attention(...): the gradients of a weighted sum of outputs against
    central differences of the 64-bit forward along random directions."""
    B, Hq, Hkv, L, d, window, sink = 1, 4, 2, 203, 64, 40, 6
    q, k, v, w = _inputs(B, Hq, Hkv, L, d, d, seed=77)
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    y = attention(*leaves, mask="window", window=window, sink=sink)
    y.backward(w.to(DEV))
    sync_status()
    _, e = _bounds(q, k, v, w, window, sink)
    rng = np.random.default_rng(5)
    x0 = [t.double().numpy() for t in (q, k, v)]

    def value(x):
        return (oracle.attention(*x, mask="window", window=window, sink=sink)[0] * w.double().numpy()).sum()
    for i, n in enumerate(("dq", "dk", "dv")):
        for _ in range(3):
            u = rng.normal(size=x0[i].shape)
            h = 1e-5
            up, dn = list(x0), list(x0)
            up[i], dn[i] = x0[i] + h * u, x0[i] - h * u
            diff = (value(up) - value(dn)) / (2 * h)
            g = leaves[i].grad.double().cpu().numpy()
            # central differences are exact to h^2 times third derivatives
            assert abs((g * u).sum() - diff) <= 1.05 * (e[n] * np.abs(u)).sum() + 1e-6 * abs(diff) + 1e-6, n


@gpu
def test_limits_agree_with_the_other_masks():
    """No sinks: bit for bit the window mask.  Sinks or a window over all keys:
    the causal mask's values."""
    q, k, v, _ = _inputs(2, 4, 2, 600, 64, 64, seed=3)
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    a = attn_fwd(q, k, v, mask="window", window=90)
    b = attn_fwd(q, k, v, mask="window", window=90, sink=0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = attn_fwd(q, k, v, mask="causal")
    for kw in (dict(window=7, sink=600), dict(window=7, sink=2 ** 31 - 1), dict(window=2 ** 31 - 1, sink=3)):
        s = attn_fwd(q, k, v, mask="window", **kw)
        sync_status()
        assert (s[0].float() - c[0].float()).abs().max() <= 2e-2 and (s[1] - c[1]).abs().max() <= 1e-4


@gpu
def test_strided_inputs_token_major():
    B, Hq, Hkv, L, d = 2, 4, 2, 333, 64
    x = synth.randn_bf16((B, L, Hq + 2 * Hkv, d), synth.generator(8))
    xd = x.to(DEV).transpose(1, 2)
    buf = torch.full((B, L, Hq + 1, d), 5.0, dtype=torch.bfloat16, device=DEV)
    out, lse = attn_fwd(xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], mask="window", window=50, sink=4,
                        out=buf[:, :, :Hq].transpose(1, 2))
    sync_status()
    assert (buf[:, :, Hq] == 5.0).all()
    t = x.transpose(1, 2)
    r, e = _bounds(t[:, :Hq], t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], None, 50, 4)
    _within(out, r["out"], e["out"], "out")
    _within(lse, r["lse"], e["lse"], "lse")


@gpu
def test_captured_training_step_and_repeatable_key_gradients():
    """Forward and backward captured into a graph replay with new inputs; dk and
    dv are the same every time."""
    B, Hq, Hkv, L, d = 1, 2, 2, 1025, 64
    kw = dict(mask="window", window=64, sink=4)
    st = [t.to(DEV) for t in _inputs(B, Hq, Hkv, L, d, d, seed=1)]
    out = torch.empty_like(st[0])
    lse = torch.empty((B, Hq, L), device=DEV)
    g = [torch.empty_like(t) for t in st[:3]]

    def run():
        attn_fwd(*st[:3], out=out, lse=lse, **kw)
        attn_bwd(*st[:3], out, st[3], lse, dq=g[0], dk=g[1], dv=g[2], **kw)
    run()
    sync_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (21, 22):
        new = _inputs(B, Hq, Hkv, L, d, d, seed=seed)
        for a, b in zip(st, new):
            a.copy_(b)
        first = None
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            if first is not None:
                assert torch.equal(first[0], g[1]) and torch.equal(first[1], g[2])
            first = (g[1].clone(), g[2].clone())
        sync_status()
        r, e = _bounds(*new, 64, 4)
        _within(out, r["out"], e["out"], "out")
        for n, t in zip(("dq", "dk", "dv"), g):
            _within(t, r[n], e[n], n)


@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("L", [100, 128, 300, 1000, 2048])
@pytest.mark.parametrize("window,sink", [(64, 4), (1, 1), (128, 128), (200, 300), (256, 4), (5000, 7), (10, 5000)])
def test_schedule_walks_each_visible_block_once(L, window, sink, d, dv):
    """fl_attn_schedule (host): the (query tile, key tile) pairs computed are
    the blocks with a visible window pair plus those with a visible sink pair
    left of the window (a block with both is walked for each); two value heads
    that share a ring (d 128) may add one window tile a query tile."""
    B, H = 1, 2
    desc = _lib.new_desc()
    desc.B, desc.Hq, desc.Hkv, desc.Lq, desc.Lk, desc.d, desc.dv = B, H, H, L, L, d, dv
    desc.mask_kind, desc.window, desc.sink = 2, window, sink
    tiles = (ctypes.c_int64 * 3)()
    assert _lib.lib().fl_attn_schedule(ctypes.byref(desc), None, tiles) == _lib.FL_OK
    nt = -(-L // 128)
    i, j = np.arange(L)[:, None], np.arange(L)[None, :]

    def blocks(vis):
        pad = np.zeros((nt * 128, nt * 128), bool)
        pad[:L, :L] = vis
        return pad.reshape(nt, 128, nt, 128).any(axis=(1, 3))
    win = blocks((j <= i) & (j > i - window))
    snk = blocks((j < sink) & (j <= i - window))
    want = B * H * int(win.sum() + snk.sum())
    if d == 64:
        # both query tiles of a unit walk the sink tiles that either needs
        pairs = np.zeros_like(snk)
        for a in range(0, nt, 2):
            pairs[a:a + 2] = snk[a:a + 2].any(0)
        want = B * H * int(win.sum() + pairs.sum())
        assert tiles[0] == want
    else:
        assert want <= tiles[0] <= want + B * H * (nt * 2 + nt * -(-min(sink, L) // 128))


@gpu
@pytest.mark.parametrize("case", [
    # (B, Hq, Hkv, L, d, dv, window, sink, score_mod)
    (1, 1, 1, 15, 128, 128, 4, 4, "softcap"), (2, 16, 4, 12, 128, 128, 3, 200, "softcap"), (3, 4, 2, 1, 64, 64, 7, 2, "none"),
    (2, 3, 3, 2, 64, 64, 1, 1, "none"), (1, 8, 1, 64, 64, 64, 5, 2, "none"), (2, 4, 2, 63, 128, 128, 20, 9, "alibi"),
    (2, 6, 2, 17, 32, 32, 6, 1, "softcap"), (40, 8, 8, 33, 64, 64, 2 ** 31 - 1, 4, "none"), (2, 4, 2, 50, 64, 128, 16, 3, "none"),
    (1, 2, 2, 64, 128, 128, 64, 64, "none"), (1, 2, 1, 48, 64, 64, 1, 1, "alibi"),
    # clusters of 2, 4 and 8 that share a group's heads, and one block for all of them
    (2, 6, 1, 31, 64, 64, 9, 2, "none"), (1, 16, 1, 64, 128, 128, 30, 4, "softcap"), (3, 12, 3, 40, 64, 128, 8, 3, "none"),
    (90, 8, 2, 20, 32, 32, 5, 1, "none"),
], ids=lambda c: "-".join(str(x) for x in c))
def test_short_sequences_keep_their_gradients_to_the_rounding(case):
    """Up to 64 tokens P and dS are not rounded to bf16 between the products: in
    two bf16 parts they keep 2^-16 of their value.  With ds, eP and eD (D from the
    scores) as above: eS = P (eD + eP) + (ds + 2^-16 + 2^-20) |dS| (+ 2^-20 P |dP
    - D| for softcap's 1 - tanh^2); dQ and dK are scale sum eS |k|, scale sum eS
    |q| off, dV sum (ds + 2^-16) P |dO|, and each is rounded once, 2^-8.  5 % for
    products of errors and the products' fp32 sums."""
    B, Hq, Hkv, L, d, dv, window, sink, mod = case
    g = synth.generator(L * 31 + d + window % 97)
    q, k = synth.randn_bf16((B, Hq, L, d), g), synth.randn_bf16((B, Hkv, L, d), g)
    v, do = synth.randn_bf16((B, Hkv, L, dv), g), synth.randn_bf16((B, Hq, L, dv), g)
    kw = dict(mask="window", window=window, sink=sink)
    slopes, cap = None, None
    if mod == "softcap":
        cap = 30.0
        kw.update(score_mod="softcap", softcap=cap)
    if mod == "alibi":
        slopes = 2.0 ** -torch.arange(1, Hq + 1, dtype=torch.float32)
        kw.update(score_mod="alibi", alibi_slopes=slopes.to(DEV))
    a = [t.to(DEV) for t in (q, k, v, do)]
    out, lse = attn_fwd(*a[:3], **kw)
    guard = [torch.full((t.numel() + 512,), 7.0, dtype=torch.bfloat16, device=DEV) for t in (q, k, v)]
    grads = [x[256:-256].view(t.shape) for x, t in zip(guard, (q, k, v))]
    got = attn_bwd(*a[:3], out, a[3], lse, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
    again = attn_bwd(*a[:3], out, a[3], lse, **kw)
    sync_status()
    for x, y in zip(got, again):
        assert torch.equal(x, y)          # no atomics: the same every time
    for x in guard:
        assert (x[:256] == 7.0).all() and (x[-256:] == 7.0).all()
    scale = 1.0 / np.sqrt(d)
    vis = oracle.visibility("window", L, L, window=window, sink=sink)
    Q, K, V, O = (t.double().numpy() for t in (q, k, v, do))
    ref = {n: np.zeros(t.shape) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    err = {n: np.zeros(t.shape) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    for b in range(B):
        for h in range(Hq):
            j = h // (Hq // Hkv)
            s = scale * (Q[b, h] @ K[b, j].T)
            mag = np.where(vis, scale * (np.abs(Q[b, h]) @ np.abs(K[b, j]).T), 0).max(1)
            t = oracle.apply_score_mod(s, mod, slope=None if slopes is None else float(slopes[h]), cap=cap)
            if mod == "alibi":
                mag = mag + abs(float(slopes[h])) * L
            P, _ = oracle.attention.__globals__["softmax_rows"](np.where(vis, t, -np.inf))
            ds = ((d + 8) * 2.0 ** -22 * mag + 2.0 ** -20 * (cap or 0.0) + 2.0 ** -18)[:, None]
            dP = O[b, h] @ V[b, j].T
            eP = 2.0 ** -22 * (dv + 8) * (np.abs(O[b, h]) @ np.abs(V[b, j]).T)
            D = (P * dP).sum(1, keepdims=True)
            eD = (P * (2 * ds * np.abs(dP) + eP)).sum(1, keepdims=True)
            slope = 1 - np.tanh(s / cap) ** 2 if mod == "softcap" else 1.0
            dS = P * (dP - D) * slope
            eS = P * (eD + eP) + (ds + 2.0 ** -16 + 2.0 ** -20) * np.abs(dS)
            if mod == "softcap":
                eS = eS + 2.0 ** -20 * P * np.abs(dP - D)
            dS[0] = eS[0] = 0
            ref["dq"][b, h], err["dq"][b, h] = scale * dS @ K[b, j], scale * eS @ np.abs(K[b, j])
            ref["dk"][b, j] += scale * dS.T @ Q[b, h]
            err["dk"][b, j] += scale * eS.T @ np.abs(Q[b, h])
            ref["dv"][b, j] += P.T @ O[b, h]
            err["dv"][b, j] += ((ds + 2.0 ** -16) * P).T @ np.abs(O[b, h])
    for n, x in zip(("dq", "dk", "dv"), got):
        e = np.abs(x.double().cpu().numpy() - ref[n])
        assert (e <= 1.05 * (err[n] + 2.0 ** -8 * np.abs(ref[n])) + 1e-30).all(), n
