"""Forward units whose two query tiles see different runs of key tiles, by any
number of tiles: document masks with a border between (or in) the two, odd
numbers of query tiles, and many units a block.  Each slot skips what the other
alone sees.

Bound: P and the result are rounded to bf16, at most 2^-8 of max |v| each, and a
score is off by ds = (d + 8) 2^-22 mag + 2^-18, mag = scale sum_c |q_c k_c| < 14 here:
2 ds < 2^-10 of max |v| and of the LSE."""
import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import attn_fwd, sync_status, synth

DEV = "cuda"

DOCS = [
    [0, 159, 188, 824, 867, 869, 955, 1056],     # the second tile sees 6 tiles more than the first
    [0, 120, 1400],                              # from the first tile's border on
    [0, 1290, 1400],                             # a long document before a short one
    [0, 1, 2, 700, 701, 2048],
    [0, 128, 256, 1900, 2050],
    [0, 900, 1100, 2000],
]


def check(out, lse, ref, v):
    ro, rl = ref
    top = float(v.abs().max())
    assert np.abs(out.double().cpu().numpy() - ro).max() <= (2.0 ** -7 + 2.0 ** -10) * top
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 2.0 ** -10


@pytest.mark.gpu
@pytest.mark.parametrize("docs", DOCS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("d,dv", [(64, 64), (32, 32), (32, 64), (64, 32), (128, 64), (128, 32), (64, 128), (128, 128)])
@pytest.mark.parametrize("doc_causal", [False, True], ids=["whole", "causal"])
def test_documents_that_part_the_slots(docs, d, dv, doc_causal):
    L = docs[-1]
    q, k, v = synth.attn_inputs(1, 1, 1, L, d, dv, seed=L + d)
    offs = torch.tensor([docs], dtype=torch.int32)
    out, lse = attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), mask="document", doc_offsets=offs.to(DEV), doc_causal=doc_causal)
    sync_status()
    check(out, lse, oracle.attention(q, k, v, mask="document", doc_offsets=offs, doc_causal=doc_causal), v)


@pytest.mark.gpu
@pytest.mark.parametrize("d,dv", [(64, 64), (32, 32), (128, 64)])
@pytest.mark.parametrize("mod", [dict(), dict(score_mod="alibi"), dict(score_mod="softcap", softcap=20.0)], ids=str)
def test_many_units_a_block_of_different_documents(d, dv, mod):
    """Units of every pattern one after another in a block, twice the same."""
    B, H = 48, 8
    L = 1100
    rng = np.random.default_rng(d)
    offs = torch.tensor(np.stack([np.concatenate(([0], np.sort(rng.choice(np.arange(1, L), 5, replace=False)), [L]))
                                  for _ in range(B)]), dtype=torch.int32)
    g = torch.Generator(device=DEV).manual_seed(d)
    q, k = (torch.randn(B, H, L, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    v = torch.randn(B, H, L, dv, generator=g, device=DEV).bfloat16()
    kw = dict(mod)
    slopes = synth.alibi_slopes(H)
    if mod.get("score_mod") == "alibi":
        kw["alibi_slopes"] = slopes.to(DEV)
    out, lse = attn_fwd(q, k, v, mask="document", doc_offsets=offs.to(DEV), **kw)
    again, _ = attn_fwd(q, k, v, mask="document", doc_offsets=offs.to(DEV), **kw)
    sync_status()
    assert torch.equal(out, again)
    doc = torch.zeros(B, L, dtype=torch.long)
    for b in range(B):
        doc[b, offs[b, 1:-1].long()] = 1
    doc = doc.cumsum(1).to(DEV)
    i = torch.arange(L, device=DEV)
    for b in range(0, B, 6):
        s = (q[b].double() @ k[b].double().transpose(-1, -2)) * d ** -0.5
        if mod.get("score_mod") == "alibi":
            s = s + slopes.double().to(DEV)[:, None, None] * (i[None] - i[:, None])
        if mod.get("score_mod") == "softcap":
            s = 20.0 * torch.tanh(s / 20.0)
        s = s.masked_fill(doc[b][:, None] != doc[b][None], float("-inf"))
        ref = torch.softmax(s, -1) @ v[b].double(), torch.logsumexp(s, -1)
        # an ALiBi bias reaches the score in fp32 of a document's length: 2^-24 1100 / 2 more
        check(out[b], lse[b], [t.cpu().numpy() for t in ref], v[b])


@pytest.mark.gpu
@pytest.mark.parametrize("L", [129, 300, 1300, 2500])
@pytest.mark.parametrize("mask", [dict(), dict(mask="causal"), dict(mask="window", window=200), dict(mask="prefix_lm", prefix=700)],
                         ids=str)
def test_odd_query_tiles_among_many_units(L, mask):
    """The last query tile of a head has no partner: its unit's second slot walks
    one tile of the ring and passes the others."""
    B, H, d = 24, 8, 64
    g = torch.Generator(device=DEV).manual_seed(L)
    q, k, v = (torch.randn(B, H, L, d, generator=g, device=DEV).bfloat16() for _ in range(3))
    out, lse = attn_fwd(q, k, v, **mask)
    again, _ = attn_fwd(q, k, v, **mask)
    sync_status()
    assert torch.equal(out, again)
    i = torch.arange(L, device=DEV)
    kind = mask.get("mask")
    vis = torch.ones(L, L, dtype=torch.bool, device=DEV) if kind is None else i[None] <= i[:, None]
    if kind == "window":
        vis &= i[None] > i[:, None] - 200
    if kind == "prefix_lm":
        vis |= i[None] < 700
    for b in range(0, B, 5):
        s = ((q[b].double() @ k[b].double().transpose(-1, -2)) * d ** -0.5).masked_fill(~vis, float("-inf"))
        check(out[b], lse[b], [(torch.softmax(s, -1) @ v[b].double()).cpu().numpy(), torch.logsumexp(s, -1).cpu().numpy()], v[b])
