"""The backward's key-tile walks when there are many more of them than blocks
that fit the GPU, so that blocks take walk after walk: the gradients of a large
batch against those of its entries alone, whose few walks get a block each.

dk and dv of a walk are summed in one order whoever does it: bit-equal (but for
the sinks' own tile, whose walk is cut by the size of the whole problem).  dq is
summed with fp32 atomics in any order, n <= 16 key tiles and their 128-key
products: the two sums differ by at most 2 n 2^-24 of the sum of magnitudes A,
and each is rounded to bf16 once (half a step, 2^-8 relative):
|difference| <= 2^-7 |dq| + 2^-19 A, A = scale sum_k |dS| |k| in 64 bits.
"""
import pytest
import torch

from flashattention_attn_fwd_gb300 import attn_bwd, attn_fwd, synth, sync_status

pytestmark = pytest.mark.gpu
DEV = "cuda"

CASES = [
    # (B, Hq, Hkv, Lq, Lk, d, kwargs)
    (12, 8, 8, 512, 512, 64, dict(mask="causal")),
    (12, 8, 8, 512, 512, 32, dict(mask="causal")),
    (10, 8, 4, 640, 640, 64, dict()),
    (40, 4, 4, 640, 640, 64, dict(mask="window", window=1)),
    (24, 4, 4, 1000, 1000, 64, dict(mask="window", window=128)),
    (24, 4, 2, 1001, 1001, 64, dict(mask="window", window=200, sink=4)),
    (24, 4, 4, 601, 601, 32, dict(mask="window", window=100, sink=130)),
    (16, 4, 4, 500, 500, 64, dict(mask="prefix_lm", prefix=150)),
    (24, 4, 4, 640, 640, 64, dict(mask="document", docs=[0, 1, 128, 300, 301, 512, 640])),
    (24, 4, 4, 640, 640, 64, dict(mask="document", doc_causal=True, docs=[0, 128, 256, 384, 400, 639, 640])),
    (12, 8, 8, 512, 512, 64, dict(mask="causal", score_mod="softcap", softcap=8.0)),
    (12, 8, 8, 512, 512, 64, dict(mask="causal", score_mod="alibi")),
    # walks of one step
    (32, 2, 2, 128, 1100, 64, dict()),
    (64, 4, 4, 4, 700, 64, dict()),
    (24, 4, 2, 100, 1300, 32, dict(score_mod="softcap", softcap=8.0)),
    # and the heads that get a block per walk
    (12, 4, 4, 512, 512, 128, dict(mask="causal")),
    (32, 2, 2, 128, 1100, 128, dict()),
]


def _magnitude(q, k, v, out, do, lse, kw, h):
    """scale sum_k |dS| |k| of one query head, 64 bits, from the scores alone:
    |dS| <= P (|dP| + |D|) bounds every mask and score transform."""
    d = q.shape[-1]
    s = (q @ k.T) / d ** 0.5
    if kw.get("score_mod") == "softcap":
        s = kw["softcap"] * torch.tanh(s / kw["softcap"])
    if kw.get("score_mod") == "alibi":
        i = torch.arange(s.shape[0], device=DEV)[:, None]
        s = s + float(kw["alibi_slopes"][h]) * (torch.arange(s.shape[1], device=DEV)[None] - i)
    # a key that the row does not see may score above the row's LSE: its weight
    # is bounded by 1, as every visible one's
    P = torch.exp(s - lse[:, None]).clamp(max=1.0)
    ds = P * ((do @ v.T).abs() + (do * out).sum(-1, keepdim=True).abs())
    return (ds @ k.abs()) / d ** 0.5


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]) + "-" + "-".join(
    str(x) for x in c[6].values() if not isinstance(x, list)))
def test_many_walks_give_the_same_gradients(case):
    B, Hq, Hkv, Lq, Lk, d, kw = case
    kw = dict(kw)
    docs = kw.pop("docs", None)
    if kw.get("score_mod") == "alibi":
        kw["alibi_slopes"] = (2.0 ** -torch.arange(1, Hq + 1, dtype=torch.float32)).to(DEV)
    g = synth.generator(B * 1000 + Lq + d)
    q = (synth.randn_bf16((B, Hq, Lq, d), g)).to(DEV)
    k, v = (synth.randn_bf16((B, Hkv, Lk, d), g).to(DEV) for _ in range(2))
    do = synth.randn_bf16((B, Hq, Lq, d), g).to(DEV)

    def variant(n):
        return kw if docs is None else dict(kw, doc_offsets=torch.tensor([docs] * n, dtype=torch.int32, device=DEV))

    out, lse = attn_fwd(q, k, v, **variant(B))

    def grads(i, j):
        a = [t[i:j].contiguous() for t in (q, k, v, out, do, lse)]
        return attn_bwd(*a, **variant(j - i))
    big = grads(0, B)
    sync_status()
    for _ in range(3):
        again = grads(0, B)
        assert torch.equal(big[1], again[1]) and torch.equal(big[2], again[2])
    own = 128 * -(-kw["sink"] // 128) if kw.get("sink") else 0   # the sinks' tiles
    for b in (0, B // 2, B - 1):
        one = grads(b, b + 1)
        for name, x, y in (("dk", big[1][b], one[1][0]), ("dv", big[2][b], one[2][0])):
            assert torch.equal(x[:, own:], y[:, own:]), name
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            fin = torch.isfinite(lse[b, h])
            A = _magnitude(q[b, h].double(), k[b, kv].double(), v[b, kv].double(), out[b, h].double(),
                           do[b, h].double(), torch.where(fin, lse[b, h], torch.zeros_like(lse[b, h])).double(), kw, h)
            x, y = big[0][b, h].double(), one[0][0, h].double()
            assert ((x - y).abs() <= 2.0 ** -7 * y.abs() + 2.0 ** -19 * A).all(), f"dq {b} {h}"
    sync_status()
