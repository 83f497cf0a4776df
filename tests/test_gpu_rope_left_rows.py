"""Rotation with positions outside the tables: their rows are left as they are in tensors
that the call is given, and zeros in those that it allocates."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import rope, rope_bwd, rope_fwd, sync_status, synth
from tests._left import dirty, reported
from tests._paged import rope_tables
from tests.test_gpu_paged import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("case", [(2, 4, 2, 6, 64, 64), (64, 8, 8, 1, 128, 64), (1, 1, 3, 40, 32, 32), (2, 8, 2, 1500, 64, 32)], ids=str)
def test_rope_positions_outside_the_tables(case, interleaved):
    B, Hq, Hk, L, d, rot = case
    g = synth.generator(1)
    q, k = (synth.randn_bf16((B, h, L, d), g).to(DEV) for h in (Hq, Hk))
    cos, sin = (t.to(DEV) for t in rope_tables(10, rot))
    pos = torch.randint(0, 10, (B, L), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    bad = torch.rand((B, L), generator=torch.Generator().manual_seed(3)) < 0.3
    bad[0, 0] = True
    pos[bad] = torch.tensor([-1, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(B * L)[:int(bad.sum())]
    kw = dict(positions=pos.to(DEV), rope_interleaved=interleaved)
    ok = ~bad[:, None].to(DEV)
    good = dict(kw, positions=pos.clamp(0, 9).to(DEV))
    for call in (rope_fwd, rope_bwd):
        wq, wk = call(q, k, cos, sin, **good)
        sync_status()
        wq, wk = (torch.where(ok[..., None], w, torch.zeros_like(w)) for w in (wq, wk))
        dirty((q.shape, q.dtype), (k.shape, k.dtype))
        a, b = call(q, k, cos, sin, **kw)
        reported()
        assert torch.equal(a, wq) and torch.equal(b, wk)
        # one given, one allocated: only the given one's rows are left
        given = torch.full_like(q, 7.0)
        dirty((k.shape, k.dtype))
        _, b = call(q, k, cos, sin, **kw, **{"q_out" if call is rope_fwd else "dq": given})
        reported()
        assert torch.equal(b, wk)
        assert torch.equal(given, torch.where(ok[..., None], wq, torch.full_like(wq, 7.0)))
        given = torch.full_like(k, 7.0)
        dirty((q.shape, q.dtype))
        a, _ = call(q, k, cos, sin, **kw, **{"k_out" if call is rope_fwd else "dk": given})
        reported()
        assert torch.equal(a, wq)
        assert torch.equal(given, torch.where(ok[..., None], wk, torch.full_like(wk, 7.0)))
        a, none = call(q, None, cos, sin, **kw)
        reported()
        assert none is None and torch.equal(a, wq)


def test_rope_autograd_with_padding_positions():
    """Finite values and gradients in the rows of padding tokens."""
    B, H, L, d = 2, 4, 50, 64
    g = synth.generator(4)
    q, k = (synth.randn_bf16((B, H, L, d), g).to(DEV).requires_grad_() for _ in range(2))
    cos, sin = (t.to(DEV) for t in rope_tables(64, d))
    pos = torch.arange(L, dtype=torch.int32).repeat(B, 1)
    pos[1, 30:] = -1
    dirty((q.shape, q.dtype), (q.shape, q.dtype), (q.shape, q.dtype), (q.shape, q.dtype))
    a, b = rope(q, k, cos, sin, positions=pos.to(DEV))
    dirty((q.shape, q.dtype), (q.shape, q.dtype))
    dq, dk = torch.autograd.grad((a, b), (q, k), (torch.ones_like(a), torch.ones_like(b)))
    reported()
    for t in (a, b, dq, dk):
        assert (t[1, :, 30:] == 0).all() and torch.isfinite(t).all() and (t[1, :, :30].abs().sum(-1) > 0).all()
