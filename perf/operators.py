"""Measured cases of the streaming-attention operators: a paged key/value
cache held in bf16 or in 4 bits, the append that rotates and stores new
tokens, the decode attention that reads it, and sliding-window attention with
sink tokens (the first keys stay visible), forward and backward.

``own = False`` computes each operator in its plain form with elementary torch
operations; ``own = True`` makes the framework's calls.  ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import random

import numpy as np
import torch

own = False

# The values of the 4-bit code (1 sign, 2 exponent, 1 mantissa bit), the low
# three bits; a block of 16 channels shares one 8-bit (e4m3) scale.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 16
SIXTH = float(np.float32(1.0) / np.float32(6.0))


# ------------------------------------------------------------------- cases

def listed():
    return [
        # append: one sequence generating one token (interactive use; latency)
        dict(name="append-1tok-e2m1", op="append", fmt="e2m1", B=1, n_min=1, n_max=1, past=700, Hq=32, Hkv=8, d=64,
             page=16, rot=64, interleaved=False, values=False, lens=1),
        # append: a serving batch, one token for each of 64 sequences
        dict(name="append-batch64-bf16", op="append", fmt="bf16", B=64, n_min=1, n_max=1, past=4096, Hq=32, Hkv=8,
             d=128, page=64, rot=128, interleaved=False, values=False, lens=2),
        # append: prompts of odd lengths, packed; the values that the 4-bit
        # cache now stands for come back for the prompts' own attention
        dict(name="append-prompts-e2m1", op="append", fmt="e2m1", B=5, n_min=900, n_max=3001, past=0, Hq=32, Hkv=8,
             d=128, page=32, rot=128, interleaved=False, values=True, lens=3),
        # append: a long prompt, rotation of half of the channels in pairs
        dict(name="append-prompt-bf16-half", op="append", fmt="bf16", B=1, n_min=16384, n_max=16384, past=0, Hq=16,
             Hkv=16, d=64, page=16, rot=32, interleaved=True, values=True, lens=4),
        # decode: one sequence, a short cache (interactive use; latency)
        dict(name="decode-1seq-e2m1", op="decode", fmt="e2m1", B=1, Lq=1, Hq=32, Hkv=8, d=64, len_min=701, len_max=701,
             page=16, mask="none", window=0, sink=0, softcap=0.0, lens=5),
        # decode: a mixed serving batch over a cache of 8192 tokens
        dict(name="decode-batch16-e2m1", op="decode", fmt="e2m1", B=16, Lq=1, Hq=32, Hkv=8, d=64, len_min=2048,
             len_max=8192, page=16, mask="none", window=0, sink=0, softcap=0.0, lens=6),
        # decode: long contexts, wide heads
        dict(name="decode-long-e2m1", op="decode", fmt="e2m1", B=12, Lq=1, Hq=32, Hkv=8, d=128, len_min=9001,
             len_max=32768, page=64, mask="causal", window=0, sink=0, softcap=0.0, lens=7),
        # decode: four drafted tokens a sequence checked at once, bf16 cache
        dict(name="decode-draft4-bf16", op="decode", fmt="bf16", B=8, Lq=4, Hq=32, Hkv=4, d=128, len_min=1500,
             len_max=16001, page=32, mask="causal", window=0, sink=0, softcap=0.0, lens=8),
        # decode: window with sinks over a long 4-bit cache
        dict(name="decode-window-sink-e2m1", op="decode", fmt="e2m1", B=32, Lq=1, Hq=16, Hkv=4, d=128, len_min=5000,
             len_max=20000, page=64, mask="window", window=1024, sink=4, softcap=0.0, lens=9),
        # training step of a small model, odd length
        dict(name="sink-train-small", op="sink", train=True, B=1, Hq=2, Hkv=2, L=301, d=64, window=64, sink=4,
             softcap=0.0),
        # training step at the benchmark's ordinary shape
        dict(name="sink-train", op="sink", train=True, B=4, Hq=16, Hkv=16, L=2048, d=64, window=256, sink=4,
             softcap=0.0),
        # long prompt, grouped heads, forward only
        dict(name="sink-prompt-gqa", op="sink", train=False, B=2, Hq=32, Hkv=8, L=8192, d=128, window=1024, sink=16,
             softcap=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("append", "decode", "sink"))
    d = rng.choice((64, 128))
    if op == "append":
        one = rng.random() < 0.5
        B = _log_int(rng, 1, 64) if one else rng.randint(1, 6)
        Hkv = rng.choice((1, 2, 4, 8))
        return dict(op=op, fmt=rng.choice(("bf16", "e2m1")), B=B, n_min=1, n_max=1 if one else _log_int(rng, 2, 2500),
                    past=_log_int(rng, 1, 8000), Hq=Hkv * rng.choice((1, 2, 4)), Hkv=Hkv, d=d,
                    page=rng.choice((16, 32, 64, 128, 256)), rot=rng.choice((d, d // 2)),
                    interleaved=rng.random() < 0.5, values=rng.random() < 0.5, lens=rng.randrange(1 << 30))
    if op == "decode":
        B = _log_int(rng, 1, 16)
        Hkv = rng.choice((1, 2, 4, 8))
        top = _log_int(rng, 1, 9000)
        mask = rng.choice(("none", "causal", "window"))
        Lq = rng.choice((1, 1, 1, 2, 3, 5))
        return dict(op=op, fmt=rng.choice(("bf16", "e2m1")), B=B, Lq=Lq, Hq=Hkv * rng.choice((1, 3, 4, 8)), Hkv=Hkv,
                    d=d, len_min=max(Lq, top // 4), len_max=max(Lq, top), page=rng.choice((16, 32, 64, 128, 256)),
                    mask=mask, window=_log_int(rng, 1, 4096) if mask == "window" else 0,
                    sink=rng.choice((0, 1, 4, 17, 130)) if mask == "window" else 0,
                    softcap=rng.choice((0.0, 0.0, 30.0)), lens=rng.randrange(1 << 30))
    Hkv = rng.choice((1, 2, 4))
    train = rng.random() < 0.6
    return dict(op=op, train=train, B=rng.randint(1, 2), Hq=Hkv * rng.choice((1, 2, 4)), Hkv=Hkv,
                L=_log_int(rng, 1, 3000 if train else 6000), d=d, window=_log_int(rng, 1, 1500),
                sink=rng.choice((1, 4, 33, 128, 200)), softcap=rng.choice((0.0, 0.0, 30.0)))


def _counts(case):
    """Lengths that a case stands for: fixed by the case, not by the seed."""
    r = random.Random(case["lens"])
    if case["op"] == "append":
        new = [r.randint(case["n_min"], case["n_max"]) for _ in range(case["B"])]
        past = [r.randint(case["past"] // 2, case["past"]) for _ in range(case["B"])]
        return new, past
    return [r.randint(case["len_min"], case["len_max"]) for _ in range(case["B"])], None


# ------------------------------------------------------------------ inputs

def _pool(case, lens, gen, filled):
    """A page pool somewhat larger than needed and a table that hands its
    pages out in random order, as a long-running server's is."""
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    need = [-(-n // page) for n in lens]
    width = max(need) + 1
    pages = sum(need) + 8
    perm = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    row = torch.tensor(need, device="cuda")
    first = torch.cumsum(row, 0) - row
    col = torch.arange(width, device="cuda")
    idx = (first[:, None] + col[None, :]).clamp_(max=pages - 1)
    table = torch.where(col[None, :] < row[:, None], perm[idx], torch.full_like(perm[idx], -1)).contiguous()
    s = {"table": table}
    if case["fmt"] == "bf16":
        make = (lambda: torch.randn(pages, Hkv, page, d, generator=gen, device="cuda").bfloat16()) if filled else \
            (lambda: torch.zeros(pages, Hkv, page, d, device="cuda", dtype=torch.bfloat16))
        s["k"], s["v"] = make(), make()
        s["k_scales"] = s["v_scales"] = None
        s["k_scale"] = s["v_scale"] = 1.0
    else:
        def codes():
            shape = (pages, Hkv, page, d // 2)
            if not filled:
                return torch.zeros(shape, device="cuda", dtype=torch.uint8)
            # rounded normal values: both nibbles from the distribution of
            # quantised activations rather than uniform codes
            mag = torch.tensor([0, 1, 1, 2, 2, 3, 3, 4, 4, 4, 5, 5, 5, 6, 6, 7], device="cuda", dtype=torch.uint8)
            lo = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
            hi = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
            lo = mag[(lo & 15).int()] | ((lo >> 4) & 8)
            hi = mag[(hi & 15).int()] | ((hi >> 4) & 8)
            return lo | (hi << 4)

        def scales(shape):
            if not filled:
                return torch.zeros(shape, device="cuda", dtype=torch.uint8)
            # e4m3 codes of block scales around 0.25 .. 0.5 (normal values)
            return torch.randint(0x26, 0x34, shape, generator=gen, device="cuda", dtype=torch.uint8)
        s["k"], s["v"] = codes(), codes()
        s["k_scales"] = scales((pages, Hkv, page, d // BLOCK))
        s["v_scales"] = scales((pages, Hkv, d // BLOCK, page))
        s["k_scale"], s["v_scale"] = 1.25, 0.75
    return s


def _rope_tables(positions, rot):
    """cos and sin of position * 10000^(-2i/rot), angles in 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)[None, :]
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "sink":
        B, Hq, Hkv, L, d = (case[k] for k in ("B", "Hq", "Hkv", "L", "d"))

        def t(H):
            return torch.randn(B, H, L, d, generator=gen, device="cuda").bfloat16()
        if case["train"]:
            s["q"], s["k"], s["v"], s["dout"] = t(Hq), t(Hkv), t(Hkv), t(Hq)
        else:
            # the projection's token-major output, seen as [B, H, L, d]
            x = torch.randn(B, L, Hq + 2 * Hkv, d, generator=gen, device="cuda").bfloat16().transpose(1, 2)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        return s
    B, Hq, Hkv, d = (case[k] for k in ("B", "Hq", "Hkv", "d"))
    if case["op"] == "append":
        new, past = _counts(case)
        total = [n + p for n, p in zip(new, past)]
        T = sum(new)
        s.update(_pool(case, total, gen, filled=False))
        s["T"] = T
        # some keys have channels far larger than the rest, as in real models
        x = torch.randn(T, Hq + 2 * Hkv, d, generator=gen, device="cuda")
        x[:, Hq:Hq + Hkv, 5::31] *= 6.0
        x = x.bfloat16()
        s["q_new"], s["k_new"], s["v_new"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["kv_len"] = torch.tensor(total, device="cuda", dtype=torch.int32)
        s["offsets"] = torch.tensor([0] + list(np.cumsum(new)), device="cuda", dtype=torch.int32)
        s["cos"], s["sin"] = _rope_tables(max(total), case["rot"])
        s["q_out"] = torch.zeros(T, Hq, d, device="cuda", dtype=torch.bfloat16)
        s["k_out"] = torch.zeros(T, Hkv, d, device="cuda", dtype=torch.bfloat16) if case["values"] else None
        s["v_out"] = torch.zeros(T, Hkv, d, device="cuda", dtype=torch.bfloat16) if case["values"] else None
    else:
        lens, _ = _counts(case)
        s.update(_pool(case, lens, gen, filled=True))
        s["kv_len"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        Lq = case["Lq"]
        s["q"] = torch.randn(B, Lq, Hq, d, generator=gen, device="cuda").bfloat16().transpose(1, 2)
        s["out"] = torch.zeros(B, Lq, Hq, d, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
        s["lse"] = torch.zeros(B, Hq, Lq, device="cuda")
    if own:
        from flashattention_attn_fwd_gb300 import PagedKVCache
        s["cache"] = PagedKVCache(s["k"], s["v"], s["k_scales"], s["v_scales"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
        if case["op"] == "decode":
            from flashattention_attn_fwd_gb300 import attn_paged_decode_workspace_size
            n = attn_paged_decode_workspace_size(s["q"], s["cache"], s["table"])
            s["workspace"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    return s


# --------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["op"] == "append":
        (_append_own if own else _append_plain)(state)
        r = {"q": state["q_out"], "k_cache": state["k"], "v_cache": state["v"]}
        if case["fmt"] == "e2m1":
            r.update(k_scales=state["k_scales"], v_scales=state["v_scales"])
        if case["values"]:
            r.update(k=state["k_out"], v=state["v_out"])
        return r
    if case["op"] == "decode":
        out, lse = (_decode_own if own else _decode_plain)(state)
        return {"out": out, "lse": lse}
    return (_sink_own if own else _sink_plain)(state)


def _mod(case):
    return dict(score_mod="softcap", softcap=case["softcap"]) if case["softcap"] else {}


def _append_own(s):
    from flashattention_attn_fwd_gb300 import kv_append
    case = s["case"]
    kv_append(s["cache"], s["k_new"], s["v_new"], s["kv_len"], s["table"], seq_offsets=s["offsets"],
              rope_cos=s["cos"], rope_sin=s["sin"], rope_interleaved=case["interleaved"], q=s["q_new"],
              q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"])


def _decode_own(s):
    from flashattention_attn_fwd_gb300 import attn_paged_decode_fwd
    case = s["case"]
    kw = dict(window=case["window"], sink=case["sink"]) if case["mask"] == "window" else {}
    return attn_paged_decode_fwd(s["q"], s["cache"], s["kv_len"], s["table"], mask=case["mask"], out=s["out"],
                                 lse=s["lse"], workspace=s["workspace"], **kw, **_mod(case))


def _sink_own(s):
    from flashattention_attn_fwd_gb300 import attn_bwd, attn_fwd
    case = s["case"]
    kw = dict(mask="window", window=case["window"], sink=case["sink"], **_mod(case))
    out, lse = attn_fwd(s["q"], s["k"], s["v"], **kw)
    if not case["train"]:
        return {"out": out, "lse": lse}
    dq, dk, dv = attn_bwd(s["q"], s["k"], s["v"], out, s["dout"], lse, **kw)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------- append, plain form

def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, d] fp32, cos and sin [T, 1, rot / 2]: each product and sum
    rounded to 32 bits once."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _quantise(x, scale):
    """Codes [.., d] and block scales [.., d / 16] of fp32 x / scale: the
    block's scale is its largest magnitude over 6 in e4m3, the codes the
    nearest 4-bit values (ties to the even code)."""
    u = (x * float(np.float32(1.0) / np.float32(scale))).unflatten(-1, (-1, BLOCK))
    s8 = (u.abs().amax(-1) * SIXTH).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    t = torch.where(s > 0, u / s, torch.zeros_like(u))
    a = t.abs()
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = code | (torch.signbit(t).to(torch.uint8) << 3)
    return code.flatten(-2), s8.view(torch.uint8)


def _value(code, s8, scale):
    """What codes [.., d] with scales [.., d / 16] stand for, fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    s = s8.view(torch.float8_e4m3fn).float()
    return (lut[code.int()].unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2) * float(np.float32(scale))


def _append_plain(s):
    case = s["case"]
    T, page, rot = s["T"], case["page"], case["rot"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"][1:].contiguous(), t, right=True)
    pos = s["kv_len"][seq] - s["offsets"][seq + 1] + t
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _rotate(s["q_new"].float(), cos, sin, rot, case["interleaved"])
    k = _rotate(s["k_new"].float(), cos, sin, rot, case["interleaved"])
    v = s["v_new"].float()
    s["q_out"].copy_(q)
    where, at = s["table"][seq, pos // page], pos % page
    if case["fmt"] == "bf16":
        s["k"][where, :, at] = k.bfloat16()
        s["v"][where, :, at] = v.bfloat16()
        if case["values"]:
            s["k_out"].copy_(k)
            s["v_out"].copy_(v)
        return
    kc, ks = _quantise(k, s["k_scale"])
    vc, vs = _quantise(v, s["v_scale"])
    s["k"][where, :, at] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    s["v"][where, :, at] = vc[..., 0::2] | (vc[..., 1::2] << 4)
    s["k_scales"][where, :, at] = ks
    s["v_scales"][where, :, :, at] = vs
    if case["values"]:
        s["k_out"].copy_(_value(kc, ks, s["k_scale"]))
        s["v_out"].copy_(_value(vc, vs, s["v_scale"]))


# ------------------------------------------------------- decode, plain form

def _gathered(s, which, S):
    """Keys or values of the first S positions of every sequence, fp32
    [B, Hkv, S, d]."""
    case = s["case"]
    page = case["page"]
    table = s["table"][:, :-(-S // page)].clamp(min=0)
    x = s[which][table].transpose(1, 2).flatten(2, 3)[:, :, :S]
    if case["fmt"] == "bf16":
        return x.float()
    sc = s[which + "_scales"][table]
    sc = sc.transpose(-1, -2) if which == "v" else sc
    sc = sc.transpose(1, 2).flatten(2, 3)[:, :, :S]
    code = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    return _value(code, sc, s[which + "_scale"])


def _decode_plain(s):
    case = s["case"]
    B, Hq, Hkv, Lq, d = (case[k] for k in ("B", "Hq", "Hkv", "Lq", "d"))
    S = max(_counts(case)[0])
    q = s["q"].float().unflatten(1, (Hkv, Hq // Hkv)).flatten(2, 3)
    x = q @ _gathered(s, "k", S).transpose(-1, -2) * (1.0 / d ** 0.5)
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    x = x.unflatten(2, (Hq // Hkv, Lq))
    j = torch.arange(S, device="cuda")
    n = s["kv_len"][:, None, None]
    p = n - Lq + torch.arange(Lq, device="cuda")[None, :, None]
    seen = (j < n).expand(B, Lq, S)
    if case["mask"] != "none":
        seen = seen & (j <= p)
    if case["mask"] == "window":
        seen = seen & ((j > p - case["window"]) | (j < case["sink"]))
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = (e / z.clamp(min=1e-37)).flatten(2, 3) @ _gathered(s, "v", S)
    s["out"].copy_(o.unflatten(2, (Hq // Hkv, Lq)).flatten(1, 2))
    s["lse"].copy_((m + torch.log(z)).squeeze(-1).flatten(1, 2))
    return s["out"], s["lse"]


# ------------------------------------------- window with sinks, plain form

def _sink_plain(s):
    case = s["case"]
    Hq, Hkv, L, d = (case[k] for k in ("Hq", "Hkv", "L", "d"))
    G, scale, cap = Hq // Hkv, 1.0 / d ** 0.5, case["softcap"]
    q = s["q"].float().unflatten(1, (Hkv, G))
    k, v = s["k"].float().unsqueeze(2), s["v"].float().unsqueeze(2)
    x = q @ k.transpose(-1, -2) * scale
    th = torch.tanh(x / cap) if cap else None
    x = cap * th if cap else x
    i = torch.arange(L, device="cuda")[:, None]
    j = torch.arange(L, device="cuda")[None, :]
    x = x.masked_fill(~((j <= i) & ((j > i - case["window"]) | (j < case["sink"]))), float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    p = p / z
    o = p @ v
    r = {"out": o.flatten(1, 2).bfloat16(), "lse": (m + torch.log(z)).squeeze(-1).flatten(1, 2)}
    if not case["train"]:
        return r
    do = s["dout"].float().unflatten(1, (Hkv, G))
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    ds = ds * (1.0 - th * th) if cap else ds
    r["dq"] = (ds @ k * scale).flatten(1, 2).bfloat16()
    r["dk"] = (ds.transpose(-1, -2) @ q).sum(2).mul(scale).bfloat16()
    r["dv"] = (p.transpose(-1, -2) @ do).sum(2).bfloat16()
    return r


# ---------------------------------------------------------- work of a pass

def work(case):
    if case["op"] == "sink":
        B, Hq, Hkv, L, d = (case[k] for k in ("B", "Hq", "Hkv", "L", "d"))
        w, t = case["window"], case["sink"]
        i = np.arange(L, dtype=np.int64)
        lo = np.maximum(i - w + 1, 0)
        pairs = B * Hq * int((i - lo + 1 + np.minimum(t, lo)).sum())
        rows_q, rows_k = B * Hq * L, B * Hkv * L
        if not case["train"]:
            return {"bytes": 2 * d * (2 * rows_q + 2 * rows_k) + 4 * rows_q, "flops": 4 * d * pairs}
        # q, dout, out, dq and k, v, dk, dv; two products forward, five back
        return {"bytes": 2 * d * (4 * rows_q + 4 * rows_k) + 4 * rows_q, "flops": 14 * d * pairs}
    Hq, Hkv, d = (case[k] for k in ("Hq", "Hkv", "d"))
    row = 2 * d if case["fmt"] == "bf16" else d // 2 + d // BLOCK  # bytes of one stored key
    if case["op"] == "append":
        new, past = _counts(case)
        T = sum(new)
        seen = max(n + p for n, p in zip(new, past))  # rotations read, shared by sequences
        b = 2 * d * T * (2 * Hq + 2 * Hkv) + 2 * row * T * Hkv + 4 * case["rot"] * min(T, seen)
        if case["values"]:
            b += 2 * 2 * d * T * Hkv
        return {"bytes": b, "flops": 3 * case["rot"] * T * (Hq + Hkv)}
    B, Lq = case["B"], case["Lq"]
    lens, _ = _counts(case)
    keys = pairs = 0
    for n in lens:
        p = [n - Lq + i for i in range(Lq)]
        if case["mask"] == "window":
            lo = [max(0, x - case["window"] + 1) for x in p]
            keys += n - lo[0] + min(case["sink"], lo[0])
            pairs += sum(x - a + 1 + min(case["sink"], a) for x, a in zip(p, lo))
        else:
            keys += n
            pairs += sum(x + 1 for x in p) if case["mask"] == "causal" else n * Lq
    return {"bytes": 2 * row * keys * Hkv + (4 * d + 4) * B * Hq * Lq, "flops": 4 * d * pairs * Hq}


# -------------------------------------------------------- 64-bit definition

def _nearest_e2m1(t):
    """Index of the nearest of the eight magnitudes, ties to the even one."""
    grid = torch.tensor(E2M1, device=t.device, dtype=torch.float64)
    dist = (t.abs()[..., None] - grid).abs()
    best = dist.amin(-1, keepdim=True)
    tied = dist <= best
    even = tied & (torch.arange(8, device=t.device) % 2 == 0)
    return torch.where(even.any(-1), even.int().argmax(-1), tied.int().argmax(-1))


def _held(x, scale):
    """The values that 4 bits hold for x [.., d] (64 bits)."""
    grid = torch.tensor(E2M1, device=x.device, dtype=torch.float64)
    u = (x / float(np.float32(scale))).unflatten(-1, (-1, BLOCK))
    s = (u.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn).double()
    t = torch.where(s > 0, u / s, torch.zeros_like(u))
    return (torch.sign(t) * grid[_nearest_e2m1(t)] * s).flatten(-2) * float(np.float32(scale))


def _exact_append(case, s):
    new, past = _counts(case)
    rot, half = case["rot"], case["rot"] // 2
    pos = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, past)])
    z = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]

    def turned(x):
        x = x.double()
        y = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half),
                                                                                        slice(half, rot))
        w = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y
    # whole numbers (codes, scales) next to a border have no 64-bit value: the
    # values that they stand for are compared instead
    r = {"q": turned(s["q_new"]), "k_cache": None, "v_cache": None}
    k, v = turned(s["k_new"]), s["v_new"].double()
    if case["fmt"] == "e2m1":
        r.update(k_scales=None, v_scales=None)
        if case["values"]:
            r.update(k=torch.cat([_held(c, s["k_scale"]) for c in k.split(512)]),
                     v=torch.cat([_held(c, s["v_scale"]) for c in v.split(512)]))
        return r
    for name, x in (("k_cache", k), ("v_cache", v)):
        c = torch.zeros(s["k"].shape, device="cuda", dtype=torch.float64)
        t0 = 0
        for b, (n, p) in enumerate(zip(new, past)):
            at = torch.arange(p, p + n, device="cuda")
            c[s["table"][b][at // case["page"]].long(), :, at % case["page"]] = x[t0:t0 + n]
            t0 += n
        r[name] = c
    if case["values"]:
        r.update(k=k, v=v)
    return r


def _exact_decode(case, s):
    B, Hq, Hkv, Lq, d, page = (case[k] for k in ("B", "Hq", "Hkv", "Lq", "d", "page"))
    G = Hq // Hkv
    out = torch.zeros(B, Hq, Lq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, Hq, Lq), float("-inf"), device="cuda", dtype=torch.float64)
    signed = torch.tensor([v for v in E2M1] + [-v for v in E2M1], device="cuda", dtype=torch.float64)

    def rows(which, b, n, h):
        pages = s["table"][b, :-(-n // page)].long()
        x = s[which][pages, h].reshape(-1, s[which].shape[-1])[:n]
        if case["fmt"] == "bf16":
            return x.double()
        lo, hi = signed[(x & 15).long()], signed[(x >> 4).long()]
        sc = s[which + "_scales"][pages, h]
        sc = (sc if which == "k" else sc.transpose(1, 2)).reshape(-1, d // BLOCK)[:n]
        sc = sc.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(BLOCK, 1)
        return torch.stack((lo, hi), -1).reshape(n, d) * sc * float(np.float32(s[which + "_scale"]))
    for b, n in enumerate(_counts(case)[0]):
        j = torch.arange(n, device="cuda")
        for h in range(Hkv):
            k, v = rows("k", b, n, h), rows("v", b, n, h)
            for i in range(Lq):
                p = n - Lq + i
                seen = torch.ones(n, device="cuda", dtype=torch.bool) if case["mask"] == "none" else j <= p
                if case["mask"] == "window":
                    seen &= (j > p - case["window"]) | (j < case["sink"])
                x = s["q"][b, h * G:(h + 1) * G, i].double() @ k[seen].T / d ** 0.5
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, -1)
                out[b, h * G:(h + 1) * G, i] = torch.softmax(x, -1) @ v[seen]
    return {"out": out, "lse": lse}


def _exact_sink(case, s):
    B, Hq, Hkv, L, d = (case[k] for k in ("B", "Hq", "Hkv", "L", "d"))
    G, w, t, cap = Hq // Hkv, case["window"], case["sink"], case["softcap"]
    out = torch.zeros(B, Hq, L, d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(B, Hq, L, device="cuda", dtype=torch.float64)
    grads = [torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in "qkv"] if case["train"] else None
    step = 1024
    for b in range(B):
        for h in range(Hq):
            q, k, v = s["q"][b, h].double(), s["k"][b, h // G].double(), s["v"][b, h // G].double()
            for r0 in range(0, L, step):
                r1 = min(L, r0 + step)
                # the sinks left of the rows' keys, then the keys themselves
                first = max(0, r0 - w + 1)
                j = torch.cat((torch.arange(min(t, first), device="cuda"), torch.arange(first, r1, device="cuda")))
                i = torch.arange(r0, r1, device="cuda")[:, None]
                x = q[r0:r1] @ k[j].T / d ** 0.5
                y = cap * torch.tanh(x / cap) if cap else x
                y = torch.where((j <= i) & ((i - j < w) | (j < t)), y, torch.full_like(y, float("-inf")))
                lse[b, h, r0:r1] = torch.logsumexp(y, -1)
                p = torch.softmax(y, -1)
                out[b, h, r0:r1] = p @ v[j]
                if grads:
                    do = s["dout"][b, h, r0:r1].double()
                    g = p * (do @ v[j].T - (do * out[b, h, r0:r1]).sum(-1, keepdim=True))
                    g = (g / torch.cosh(x / cap) ** 2 if cap else g) / d ** 0.5
                    grads[0][b, h, r0:r1] = g @ k[j]
                    grads[1][b, h // G].index_add_(0, j, g.T @ q[r0:r1])
                    grads[2][b, h // G].index_add_(0, j, p.T @ do)
    r = {"out": out, "lse": lse}
    if grads:
        r.update(dq=grads[0], dk=grads[1], dv=grads[2])
    return r


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "sink": _exact_sink}[case["op"]](case, s)
