"""Measured cases of the operators around long prompts: attention of chunks of
new tokens over the paged key/value cache, the read-back of what the cache
holds, the rotation of queries and keys with its gradient, and the rotation's
tables for scaled long contexts.

``own = False`` computes each operator in its plain form with elementary torch
operations; ``own = True`` makes the framework's calls.  ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

# The values of the 4-bit code (1 sign, 2 exponent, 1 mantissa bit), the low
# three bits; a block of 16 channels shares one 8-bit (e4m3) scale.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 16


# ------------------------------------------------------------------- cases

def _prefill(name, fmt, B, new, past, Hq, Hkv, d, page, lens, mask="causal", window=0, sink=0, score="none",
             softcap=0.0):
    c = dict(op="prefill", fmt=fmt, B=B, n_min=new[0], n_max=new[1], past_min=past[0], past_max=past[1], Hq=Hq,
             Hkv=Hkv, d=d, page=page, mask=mask, window=window, sink=sink, score=score, softcap=softcap, lens=lens)
    return dict(name=name, **c) if name else c


def _read(name, fmt, B, n, Hkv, d, page, lens):
    c = dict(op="read", fmt=fmt, B=B, n_min=n[0], n_max=n[1], Hkv=Hkv, d=d, page=page, lens=lens)
    return dict(name=name, **c) if name else c


def _rope(name, B, L, Hq, Hkv, d, rot, interleaved, given, train):
    c = dict(op="rope", B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, rot=rot, interleaved=interleaved, given=given, train=train)
    return dict(name=name, **c) if name else c


def _tables(name, positions, rot, base, scaling, factor, original):
    c = dict(op="tables", positions=positions, rot=rot, base=base, scaling=scaling, factor=factor, original=original)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one sequence's next 64 tokens over a short past (interactive use; latency)
        _prefill("prefill-chunk64-bf16", "bf16", 1, (64, 64), (700, 700), 32, 8, 64, 16, 1),
        # a serving batch whose sequences bring chunks of all lengths, single tokens among them
        _prefill("prefill-mixed-e2m1", "e2m1", 16, (1, 512), (2048, 8192), 32, 8, 64, 16, 2),
        # whole prompts of odd lengths, packed
        _prefill("prefill-prompts-bf16", "bf16", 5, (900, 3001), (0, 0), 32, 8, 128, 32, 3),
        # the last chunk of a long document
        _prefill("prefill-long-bf16", "bf16", 1, (2048, 2048), (30720, 30720), 32, 8, 128, 64, 4),
        # streaming: window with sinks over a long 4-bit cache
        _prefill("prefill-window-sink-e2m1", "e2m1", 4, (1024, 1024), (4000, 19000), 16, 4, 128, 64, 5,
                 mask="window", window=1024, sink=4),
        # one sequence leaves the pool (latency)
        _read("read-1seq-e2m1", "e2m1", 1, (701, 701), 8, 64, 16, 6),
        # a batch of long sequences leaves the pool
        _read("read-batch-e2m1", "e2m1", 12, (5001, 20000), 8, 128, 64, 7),
        # one new token of every sequence of a batch, each at its own position (latency)
        _rope("rope-batch64-1tok", 64, 1, 32, 8, 128, 128, False, True, False),
        # training step at the benchmark's ordinary shape: rotation and its gradient
        _rope("rope-train", 4, 2048, 16, 16, 64, 64, False, False, True),
        # long prompt, grouped heads, half of the channels in pairs
        _rope("rope-prompt-half-pairs", 2, 8192, 32, 8, 128, 64, True, True, False),
        # tables of a short context, plain
        _tables("tables-4096", 4096, 64, 10000.0, "none", 1.0, 4096),
        # tables of a context stretched 16 times, by parts
        _tables("tables-131072-by-parts", 131072, 128, 500000.0, "by_parts", 16.0, 8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "read", "rope", "tables"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    fmt = rng.choice(("bf16", "e2m1"))
    if op == "prefill":
        top = _log_int(rng, 1, 1500)
        past = _log_int(rng, 1, 6000) - 1
        mask = rng.choice(("causal", "causal", "window", "none"))
        score = rng.choice(("none", "none", "softcap", "alibi"))
        return _prefill(None, fmt, rng.randint(1, 6), (max(1, top // 4), top), (past // 2, past),
                        Hkv * rng.choice((1, 3, 4, 8)), Hkv, d, page, rng.randrange(1 << 30), mask=mask,
                        window=_log_int(rng, 1, 3000) if mask == "window" else 0,
                        sink=rng.choice((0, 1, 4, 17, 130)) if mask == "window" else 0, score=score,
                        softcap=30.0 if score == "softcap" else 0.0)
    if op == "read":
        top = _log_int(rng, 1, 16000)
        return _read(None, fmt, rng.randint(1, 12), (max(1, top // 4), top), Hkv, d, page, rng.randrange(1 << 30))
    if op == "rope":
        L = _log_int(rng, 1, 8000)
        return _rope(None, rng.randint(1, 64) if L < 100 else rng.randint(1, 3), L, Hkv * rng.choice((1, 3, 4)), Hkv, d,
                     rng.choice((d, d // 2)), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.6)
    scaling = rng.choice(("none", "linear", "ntk", "by_parts"))
    return _tables(None, _log_int(rng, 1, 131072), rng.choice((16, 32, 64, 128)), rng.choice((10000.0, 500000.0)),
                   scaling, 1.0 if scaling == "none" else rng.choice((2.0, 4.0, 7.5, 16.0)), rng.choice((2048, 8192)))


def _counts(case):
    """Lengths that a case stands for: fixed by the case, not by the seed."""
    r = random.Random(case["lens"])
    new = [r.randint(case["n_min"], case["n_max"]) for _ in range(case["B"])]
    past = [r.randint(case["past_min"], case["past_max"]) for _ in range(case["B"])] if case["op"] == "prefill" else \
        [0] * case["B"]
    return new, past


# ------------------------------------------------------------------ inputs

def _pool(case, lens, gen):
    """A filled page pool somewhat larger than needed and a table that hands
    its pages out in random order, as a long-running server's is."""
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    need = [-(-n // page) for n in lens]
    width = max(need) + 1
    pages = sum(need) + 8
    perm = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    row = torch.tensor(need, device="cuda")
    first = torch.cumsum(row, 0) - row
    col = torch.arange(width, device="cuda")
    idx = (first[:, None] + col[None, :]).clamp_(max=pages - 1)
    s = {"table": torch.where(col[None, :] < row[:, None], perm[idx], torch.full_like(perm[idx], -1)).contiguous()}
    if case["fmt"] == "bf16":
        s["k"], s["v"] = (torch.randn(pages, Hkv, page, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
        s["k_scales"] = s["v_scales"] = None
        s["k_scale"] = s["v_scale"] = 1.0
        return s

    def codes():
        # rounded normal values: both nibbles from the distribution of
        # quantised activations rather than uniform codes
        shape = (pages, Hkv, page, d // 2)
        mag = torch.tensor([0, 1, 1, 2, 2, 3, 3, 4, 4, 4, 5, 5, 5, 6, 6, 7], device="cuda", dtype=torch.uint8)
        both = torch.cat([mag, mag | 8])
        pair = (both[:, None] << 4 | both[None, :]).flatten()  # of 10 random bits
        r = torch.randint(0, 1024, shape, generator=gen, device="cuda", dtype=torch.int16)
        return pair[r.int()]

    def scales(shape):
        # e4m3 codes of block scales around 0.25 .. 0.5 (normal values)
        return torch.randint(0x26, 0x34, shape, generator=gen, device="cuda", dtype=torch.uint8)
    s["k"], s["v"] = codes(), codes()
    s["k_scales"] = scales((pages, Hkv, page, d // BLOCK))
    s["v_scales"] = scales((pages, Hkv, d // BLOCK, page))
    s["k_scale"], s["v_scale"] = 1.25, 0.75
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "tables":
        # the context length and the frequencies' parameters are the input; a
        # server that serves several stretches computes each anew
        s["amplitude"] = 1.0 + (int(seed) % 97) / 1024.0
        half = case["rot"] // 2
        s["cos"], s["sin"] = (torch.zeros(case["positions"], half, device="cuda") for _ in range(2))
        return s
    if op == "rope":
        B, L, Hq, Hkv, d = (case[k] for k in ("B", "L", "Hq", "Hkv", "d"))
        # the projection's token-major output, seen as [B, H, L, d]
        x = torch.randn(B, L, Hq + 2 * Hkv, d, generator=gen, device="cuda").bfloat16().transpose(1, 2)
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
        if case["train"]:
            s["dq"] = torch.randn(B, Hq, L, d, generator=gen, device="cuda").bfloat16()
            s["dk"] = torch.randn(B, Hkv, L, d, generator=gen, device="cuda").bfloat16()
        span = 2 * L + 100
        s["cos"], s["sin"] = _rope_tables(span, case["rot"])
        s["positions"] = None
        if case["given"]:  # every sequence starts somewhere
            start = torch.randint(0, span - L + 1, (B, 1), generator=gen, device="cuda")
            s["positions"] = (start + torch.arange(L, device="cuda")).int()
        return s
    new, past = _counts(case)
    total = [n + p for n, p in zip(new, past)]
    T = sum(new)
    s.update(_pool(case, total, gen))
    s["T"] = T
    s["kv_len"] = torch.tensor(total, device="cuda", dtype=torch.int32)
    s["offsets"] = torch.tensor([0] + list(np.cumsum(new)), device="cuda", dtype=torch.int32)
    Hkv, d = case["Hkv"], case["d"]
    if op == "read":
        s["k_out"], s["v_out"] = (torch.zeros(T, Hkv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    else:
        Hq = case["Hq"]
        # what kv_append leaves: rotated queries, token-major
        s["q"] = torch.randn(T, Hq, d, generator=gen, device="cuda").bfloat16()
        s["out"] = torch.zeros(T, Hq, d, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros(T, Hq, device="cuda")
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq) if case["score"] == "alibi" else None
    if own:
        from flashattention_attn_fwd_gb300 import PagedKVCache
        s["cache"] = PagedKVCache(s["k"], s["v"], s["k_scales"], s["v_scales"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
        if op == "prefill":
            from flashattention_attn_fwd_gb300 import attn_paged_prefill_workspace_size
            n = attn_paged_prefill_workspace_size(s["q"], s["cache"], s["table"])
            s["workspace"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    return s


def _rope_tables(positions, rot):
    """cos and sin of position * 10000^(-2i/rot), angles in 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)[None, :]
    return a.cos().float(), a.sin().float()


# --------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    return {"prefill": _prefill_own if own else _prefill_plain, "read": _read_own if own else _read_plain,
            "rope": _rope_own if own else _rope_plain, "tables": _tables_own if own else _tables_plain}[op](state)


def _prefill_own(s):
    from flashattention_attn_fwd_gb300 import attn_paged_prefill_fwd
    case = s["case"]
    kw = dict(window=case["window"], sink=case["sink"]) if case["mask"] == "window" else {}
    if case["score"] == "softcap":
        kw.update(score_mod="softcap", softcap=case["softcap"])
    elif case["score"] == "alibi":
        kw.update(score_mod="alibi", alibi_slopes=s["slopes"])
    out, lse = attn_paged_prefill_fwd(s["q"], s["cache"], s["kv_len"], s["table"], seq_offsets=s["offsets"],
                                      mask=case["mask"], out=s["out"], lse=s["lse"], workspace=s["workspace"], **kw)
    return {"out": out, "lse": lse}


def _read_own(s):
    from flashattention_attn_fwd_gb300 import kv_read
    k, v = kv_read(s["cache"], s["kv_len"], s["table"], s["T"], seq_offsets=s["offsets"], k_out=s["k_out"],
                   v_out=s["v_out"])
    return {"k": k, "v": v}


def _rope_own(s):
    from flashattention_attn_fwd_gb300 import rope_bwd, rope_fwd
    case = s["case"]
    kw = dict(positions=s["positions"], rope_interleaved=case["interleaved"])
    q, k = rope_fwd(s["q"], s["k"], s["cos"], s["sin"], **kw)
    r = {"q": q, "k": k}
    if case["train"]:
        r["dq"], r["dk"] = rope_bwd(s["dq"], s["dk"], s["cos"], s["sin"], **kw)
    return r


def _tables_own(s):
    from flashattention_attn_fwd_gb300 import rope_tables
    case = s["case"]
    cos, sin = rope_tables(case["positions"], case["rot"], base=case["base"], scaling=case["scaling"],
                           factor=case["factor"], original=case["original"], amplitude=s["amplitude"], cos=s["cos"],
                           sin=s["sin"])
    return {"cos": cos, "sin": sin}


# ------------------------------------------------------- prefill, plain form

def _value(code, s8, scale):
    """What codes [.., d] with scales [.., d / 16] stand for, fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    sc = s8.contiguous().view(torch.float8_e4m3fn).float()
    return (lut[code.int()].unflatten(-1, (-1, BLOCK)) * sc[..., None]).flatten(-2) * float(np.float32(scale))


def _held_rows(s, which, b, n):
    """Keys or values of the first n positions of sequence b, fp32 [Hkv, n, d]."""
    case = s["case"]
    pages = s["table"][b, :-(-n // case["page"])]
    x = s[which][pages].transpose(0, 1).flatten(1, 2)[:, :n]
    if case["fmt"] == "bf16":
        return x.float()
    sc = s[which + "_scales"][pages]
    sc = (sc.transpose(-1, -2) if which == "v" else sc).transpose(0, 1).flatten(1, 2)[:, :n]
    return _value(torch.stack((x & 15, x >> 4), -1).flatten(-2), sc, s[which + "_scale"])


def _prefill_plain(s):
    case = s["case"]
    Hq, Hkv, d = (case[k] for k in ("Hq", "Hkv", "d"))
    G = Hq // Hkv
    new, past = _counts(case)
    t0 = 0
    for b, (n, p0) in enumerate(zip(new, past)):
        S = n + p0
        k, v = _held_rows(s, "k", b, S), _held_rows(s, "v", b, S)
        j = torch.arange(S, device="cuda")
        step = max(1, (1 << 28) // (Hq * S))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            q = s["q"][t0 + r0:t0 + r1].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3).flatten(1, 2)
            x = (q @ k.transpose(-1, -2) * (1.0 / d ** 0.5)).unflatten(1, (G, r1 - r0))
            p = p0 + torch.arange(r0, r1, device="cuda")[:, None]
            if case["score"] == "softcap":
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            elif case["score"] == "alibi":
                x = x + s["slopes"].view(Hkv, G, 1, 1) * (j - p)
            if case["mask"] != "none":
                seen = j <= p
                if case["mask"] == "window":
                    seen = seen & ((j > p - case["window"]) | (j < case["sink"]))
                x = x.masked_fill(~seen, float("-inf"))
            m = x.amax(-1, keepdim=True)
            e = torch.exp(x - m)
            z = e.sum(-1, keepdim=True)
            o = (e / z).flatten(1, 2) @ v
            s["out"][t0 + r0:t0 + r1] = o.unflatten(1, (G, r1 - r0)).permute(2, 0, 1, 3).flatten(1, 2).bfloat16()
            s["lse"][t0 + r0:t0 + r1] = (m + torch.log(z)).squeeze(-1).permute(2, 0, 1).flatten(1, 2)
        t0 += n
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------ the others, in plain form

def _read_plain(s):
    case = s["case"]
    page = case["page"]
    t = torch.arange(s["T"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"][1:].contiguous(), t, right=True)
    pos = s["kv_len"][seq] - s["offsets"][seq + 1] + t
    where, at = s["table"][seq, pos // page], pos % page
    for which, out in (("k", s["k_out"]), ("v", s["v_out"])):
        x = s[which][where, :, at]
        if case["fmt"] == "bf16":
            out.copy_(x)
            continue
        sc = s["k_scales"][where, :, at] if which == "k" else s["v_scales"][where, :, :, at]
        out.copy_(_value(torch.stack((x & 15, x >> 4), -1).flatten(-2), sc, s[which + "_scale"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _turn(x, cos, sin, rot, interleaved):
    """x [B, H, L, d], cos and sin [B or 1, 1, L, rot / 2]: rotated in fp32,
    each product and sum rounded once, then rounded to bf16."""
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1).bfloat16()


def _rope_plain(s):
    case = s["case"]
    rot, inter = case["rot"], case["interleaved"]
    at = slice(0, case["L"]) if s["positions"] is None else s["positions"]
    cos, sin = s["cos"][at], s["sin"][at]
    cos, sin = (x.unsqueeze(1) if x.dim() == 3 else x for x in (cos, sin))
    r = {"q": _turn(s["q"], cos, sin, rot, inter), "k": _turn(s["k"], cos, sin, rot, inter)}
    if case["train"]:
        r["dq"], r["dk"] = _turn(s["dq"], cos, -sin, rot, inter), _turn(s["dk"], cos, -sin, rot, inter)
    return r


# turns of a pair of channels within the original context between which the
# scaling by parts goes from interpolated to left alone
LOW_TURNS, HIGH_TURNS = 1.0, 32.0


def _tables_plain(s):
    case = s["case"]
    rot, f = case["rot"], case["factor"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    base = case["base"] * f ** (rot / (rot - 2)) if case["scaling"] == "ntk" else case["base"]
    inv = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        inv = inv / f
    elif case["scaling"] == "by_parts":
        g = ((case["original"] * inv / (2.0 * math.pi) - LOW_TURNS) / (HIGH_TURNS - LOW_TURNS)).clamp(0.0, 1.0)
        inv = inv * (g + (1.0 - g) / f)
    a = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * inv
    s["cos"].copy_(a.cos() * s["amplitude"])
    s["sin"].copy_(a.sin() * s["amplitude"])
    return {"cos": s["cos"], "sin": s["sin"]}


# ---------------------------------------------------------- work of a pass

def work(case):
    op = case["op"]
    if op == "tables":
        cells = case["positions"] * case["rot"] // 2
        return {"bytes": 8 * cells, "flops": 2 * cells}
    if op == "rope":
        B, L, d, rot = (case[k] for k in ("B", "L", "d", "rot"))
        rows = B * L * (case["Hq"] + case["Hkv"]) * (2 if case["train"] else 1)
        # rows in and out, a table row for each position once
        spots = min(B * L, 2 * L + 100) if case["given"] else L
        return {"bytes": 4 * d * rows + 4 * rot * spots + (4 * B * L if case["given"] else 0), "flops": 3 * rot * rows}
    Hkv, d = case["Hkv"], case["d"]
    row = 2 * d if case["fmt"] == "bf16" else d // 2 + d // BLOCK  # bytes of one stored key
    new, past = _counts(case)
    T = sum(new)
    if op == "read":
        return {"bytes": 2 * (row + 2 * d) * T * Hkv, "flops": 2 * d * T * Hkv if case["fmt"] == "e2m1" else 0}
    keys = pairs = 0
    for n, p0 in zip(new, past):
        p = np.arange(p0, p0 + n, dtype=np.int64)
        if case["mask"] == "window":
            lo = np.maximum(0, p - case["window"] + 1)
            keys += int(n + p0 - lo[0] + min(case["sink"], lo[0]))
            pairs += int((p - lo + 1 + np.minimum(case["sink"], lo)).sum())
        else:
            keys += n + p0
            pairs += int((p + 1).sum()) if case["mask"] == "causal" else n * (n + p0)
    return {"bytes": 2 * row * keys * Hkv + (4 * d + 4) * T * case["Hq"], "flops": 4 * d * pairs * case["Hq"]}


# -------------------------------------------------------- 64-bit definition

def _rows64(case, s, which, b, h, n):
    """Keys or values [n, d] of head h of sequence b."""
    pages = s["table"][b, :-(-n // case["page"])].long()
    x = s[which][pages, h].reshape(-1, s[which].shape[-1])[:n]
    if case["fmt"] == "bf16":
        return x.double()
    signed = torch.tensor(list(E2M1) + [-v for v in E2M1], device="cuda", dtype=torch.float64)
    sc = s[which + "_scales"][pages, h]
    sc = (sc if which == "k" else sc.transpose(1, 2)).reshape(-1, case["d"] // BLOCK)[:n]
    sc = sc.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(BLOCK, 1)
    both = torch.stack((signed[(x & 15).long()], signed[(x >> 4).long()]), -1).reshape(n, case["d"])
    return both * sc * float(np.float32(s[which + "_scale"]))


def _exact_prefill(case, s):
    Hq, Hkv, d = (case[k] for k in ("Hq", "Hkv", "d"))
    G, w, t = Hq // Hkv, case["window"], case["sink"]
    new, past = _counts(case)
    out = torch.zeros(sum(new), Hq, d, device="cuda", dtype=torch.float64)
    lse = torch.zeros(sum(new), Hq, device="cuda", dtype=torch.float64)
    t0 = 0
    for b, (n, p0) in enumerate(zip(new, past)):
        for h in range(Hkv):
            k, v = _rows64(case, s, "k", b, h, n + p0), _rows64(case, s, "v", b, h, n + p0)
            for r0 in range(0, n, 512):
                r1 = min(n, r0 + 512)
                end = n + p0 if case["mask"] == "none" else p0 + r1
                j = torch.arange(end, device="cuda")
                if case["mask"] == "window":  # the sinks left of the rows' keys, then the keys themselves
                    first = max(0, p0 + r0 - w + 1)
                    j = torch.cat((j[:min(t, first)], j[first:]))
                i = torch.arange(p0 + r0, p0 + r1, device="cuda")[:, None]
                for g in range(h * G, (h + 1) * G):
                    x = s["q"][t0 + r0:t0 + r1, g].double() @ k[j].T / d ** 0.5
                    if case["score"] == "softcap":
                        x = case["softcap"] * torch.tanh(x / case["softcap"])
                    elif case["score"] == "alibi":
                        x = x - float(s["slopes"][g]) * (i - j).double()
                    if case["mask"] != "none":
                        ok = (j <= i) & ((i - j < w) | (j < t)) if case["mask"] == "window" else j <= i
                        x = torch.where(ok, x, torch.full_like(x, float("-inf")))
                    lse[t0 + r0:t0 + r1, g] = torch.logsumexp(x, -1)
                    out[t0 + r0:t0 + r1, g] = torch.softmax(x, -1) @ v[j]
        t0 += n
    return {"out": out, "lse": lse}


def _exact_read(case, s):
    new, _ = _counts(case)
    return {w: torch.cat([torch.stack([_rows64(case, s, w, b, h, n) for h in range(case["Hkv"])], 1)
                          for b, n in enumerate(new)]) for w in ("k", "v")}


def _exact_rope(case, s):
    rot, L = case["rot"], case["L"]
    at = torch.arange(L, device="cuda").expand(case["B"], L) if s["positions"] is None else s["positions"].long()
    z = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2),
                                                                                    slice(rot // 2, rot))

    def turned(x, z):
        x = x.double()
        y = x.clone()
        u = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = u.real, u.imag
        return y
    r = {"q": turned(s["q"], z), "k": turned(s["k"], z)}
    if case["train"]:
        r.update(dq=turned(s["dq"], z.conj()), dk=turned(s["dk"], z.conj()))
    return r


def _exact_tables(case, s):
    rot, f = case["rot"], case["factor"]
    inv = np.empty(rot // 2)
    for i in range(rot // 2):
        x = math.exp(-2.0 * i / rot * math.log(case["base"]))
        if case["scaling"] == "linear":
            x /= f
        elif case["scaling"] == "ntk":
            x *= math.exp(-2.0 * i / (rot - 2) * math.log(f))
        elif case["scaling"] == "by_parts":
            turns = case["original"] * x / (2.0 * math.pi)
            keep = min(max((turns - LOW_TURNS) / (HIGH_TURNS - LOW_TURNS), 0.0), 1.0)
            x = keep * x + (1.0 - keep) * x / f
        inv[i] = x
    a = torch.arange(case["positions"], device="cuda", dtype=torch.float64)[:, None] * torch.from_numpy(inv).cuda()
    z = torch.polar(torch.full_like(a, s["amplitude"]), a)
    return {"cos": z.real, "sin": z.imag}


def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_prefill, "read": _exact_read, "rope": _exact_rope, "tables": _exact_tables}[case["op"]](
        case, s)
