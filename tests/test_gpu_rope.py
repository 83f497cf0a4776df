"""GPU tests of the rotary positions: rotation and its gradient bit for bit
against the 32-bit steps (each product and sum rounded once, then bf16), the
gradient also against differences, and the tables against 64 bits.

Tables' bound.  The angle's rest, at most a quarter of a half turn, is rounded to
fp32 (2^-27 half turns) after its fraction of a turn was cut to 32 bits (2^-32
turns): pi 2^-27 + 2 pi 2^-32 < 2.5e-8.  The step's fp64 value carries at most 4
roundings of 2^-53 (power, products, quotient), times the angle, which is at most the
position: 2^-51 pos; cut at 2^-64 turns it adds 2 pi 2^-64 pos.  The two
polynomials are within 9e-8, less than two units of 2^-24 (tests/test_turn_poly.py;
fused steps round less), the amplitude's product rounds by 2^-24: 3 x 2^-24."""
import math

import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import (FlattnError, attention, rope, rope_bwd, rope_fwd, rope_tables, sync_status,
                                           synth)
from tests._paged import rope_tables as host_tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


def turned(x, cos, sin, pos, interleaved, sign=1.0):
    """The 32-bit steps on x [B, H, L, d], positions [B, L]."""
    out = []
    for b in range(x.shape[0]):
        c, s = cos[pos[b]], sign * sin[pos[b]]
        y = oracle.rotate(x[b].transpose(0, 1).float().numpy(), c.numpy(), s.numpy(), interleaved, dtype=np.float32)
        out.append(torch.from_numpy(y).bfloat16().transpose(0, 1))
    return torch.stack(out)


CASES = [
    # B, Hq, Hk, L, d, rope_dim
    (1, 1, 0, 1, 32, 32),
    (2, 3, 1, 5, 32, 16),
    (64, 8, 2, 1, 64, 64),
    (2, 8, 8, 301, 64, 32),
    (3, 5, 1, 77, 128, 128),
    (1, 32, 8, 130, 128, 48),
    (1, 2, 2, 5000, 64, 64),
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("given", [False, True], ids=["from0", "given"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotation_and_gradient_bit_for_bit(case, given, interleaved):
    B, Hq, Hk, L, d, rot = case
    g = synth.generator(L + d)
    # token-major, as a projection leaves it
    x = synth.randn_bf16((B, L, Hq + Hk, d), g).transpose(1, 2)
    cos, sin = host_tables(2 * L + 7, rot)
    pos = torch.randint(0, 2 * L + 7, (B, L), generator=torch.Generator().manual_seed(L), dtype=torch.int32)
    kw = dict(rope_interleaved=interleaved, positions=pos.to(DEV) if given else None)
    xd, c, s = x.to(DEV), cos.to(DEV), sin.to(DEV)
    at = pos.long() if given else torch.arange(L).expand(B, L)
    q, k = rope_fwd(xd[:, :Hq], xd[:, Hq:] if Hk else None, c, s, **kw)
    assert q.is_contiguous()
    assert torch.equal(q.cpu(), turned(x[:, :Hq], cos, sin, at, interleaved))
    assert (k is None) == (Hk == 0)
    if Hk:
        assert k.is_contiguous() and torch.equal(k.cpu(), turned(x[:, Hq:], cos, sin, at, interleaved))
    # the gradient, into the token-major layout
    room = torch.full((B, L, Hq + Hk + 1, d), 7.0, device=DEV, dtype=torch.bfloat16)
    gq, gk = room.transpose(1, 2)[:, :Hq], room.transpose(1, 2)[:, Hq:Hq + Hk] if Hk else None
    rope_bwd(q, k, c, s, dq=gq, dk=gk, **kw)
    sync_status()
    assert torch.equal(gq.cpu(), turned(q.cpu(), cos, sin, at, interleaved, -1.0))
    if Hk:
        assert torch.equal(gk.cpu(), turned(k.cpu(), cos, sin, at, interleaved, -1.0))
    assert (room[:, :, Hq + Hk] == 7).all()


def test_in_place_shared_positions_and_another_stream():
    B, H, L, d = 3, 4, 50, 64
    x = synth.randn_bf16((B, H, L, d), synth.generator(1))
    cos, sin = host_tables(200, d)
    pos = (torch.arange(L) * 3 + 20).int()
    y, c, s, p = x.to(DEV), cos.to(DEV), sin.to(DEV), pos.to(DEV)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, k = rope_fwd(y, None, c, s, positions=p, q_out=y, stream=st)
    st.synchronize()
    sync_status()
    assert q is y and k is None
    assert torch.equal(y.cpu(), turned(x, cos, sin, pos.long().expand(B, L), False))


def test_the_gradient_is_that_of_the_definition():
    """Against differences of the 64-bit definition: dq = J^T dy, J columns by
    differences of a linear map (exact but for rounding to bf16, 2^-8 of the
    pair's size)."""
    B, H, L, d, rot = 1, 2, 7, 64, 32
    cos, sin = host_tables(L, rot)
    dy = synth.randn_bf16((B, H, L, d), synth.generator(2))
    for inter in (False, True):
        dq, _ = rope_bwd(dy.to(DEV), None, cos.to(DEV), sin.to(DEV), rope_interleaved=inter)
        sync_status()
        want = np.zeros((H, L, d))
        for c in range(d):
            e = np.zeros((L, H, d))
            e[:, :, c] = 1.0
            J = oracle.rotate(e, cos.numpy(), sin.numpy(), inter)          # column c of the turn, by token
            want[:, :, c] = np.einsum("lhd,hld->hl", J, dy[0].double().numpy())
        size = np.sqrt(2.0) * np.abs(dy[0].double().numpy()).max(-1, keepdims=True)
        assert (np.abs(dq[0].double().cpu().numpy() - want) <= 2.0 ** -8 * size).all()


def test_autograd_through_rope_and_attention():
    """rope -> attention -> loss: gradients of the unrotated q and k against the
    64-bit chain (attention's gradient tolerance, turned)."""
    B, H, L, d = 1, 2, 64, 64
    g = synth.generator(3)
    x = synth.randn_bf16((B, L, 3 * H, d), g).to(DEV).requires_grad_()
    cos, sin = host_tables(L, d)
    q, k, v = (x.transpose(1, 2)[:, i * H:(i + 1) * H] for i in range(3))
    qr, kr = rope(q, k, cos.to(DEV), sin.to(DEV))
    out = attention(qr, kr, v.contiguous(), mask="causal")
    dout = synth.randn_bf16((B, H, L, d), g)
    out.backward(dout.to(DEV))
    sync_status()
    at = torch.arange(L)[None]
    rq, rk = (turned(t.detach().cpu(), cos, sin, at, False) for t in (q, k))
    gq, gk, gv = oracle.attention_backward(rq, rk, v.detach().cpu(), dout, mask="causal")
    back = lambda t: np.swapaxes(oracle.rotate(np.swapaxes(t[0], 0, 1), cos.numpy(), -sin.numpy(), False), 0, 1)  # noqa: E731
    got = x.grad.transpose(1, 2)[0].double().cpu().numpy()
    for i, want in enumerate((back(gq), back(gk), gv[0])):
        err = got[i * H:(i + 1) * H] - want
        assert np.linalg.norm(err) <= 2.5e-2 * np.linalg.norm(want)
        assert np.abs(err).max() <= 5e-2 * np.abs(want).max()
    # an expanded gradient (of a sum) has zero strides
    qr, kr = rope(q, k, cos.to(DEV), sin.to(DEV))
    dq, = torch.autograd.grad(qr.sum() + 0 * kr.sum(), q)
    sync_status()
    assert torch.equal(dq.cpu(), turned(torch.ones(B, H, L, d).bfloat16(), cos, sin, at, False, -1.0))


def test_positions_outside_the_tables_are_left_and_reported():
    x = synth.randn_bf16((2, 2, 6, 64), synth.generator(5))
    cos, sin = host_tables(10, 64)
    pos = torch.tensor([[0, -1, 9, 10, 2 ** 31 - 1, 3], [1, 2, 3, 4, 5, -2 ** 31]], dtype=torch.int32)
    y = torch.full((2, 2, 6, 64), 7.0, device=DEV, dtype=torch.bfloat16)
    rope_fwd(x.to(DEV), None, cos.to(DEV), sin.to(DEV), positions=pos.to(DEV), q_out=y)
    with pytest.raises(FlattnError) as e:
        sync_status()
    assert e.value.status == 6
    ok = (pos >= 0) & (pos < 10)
    want = turned(x, cos, sin, pos.clamp(0, 9).long(), False)
    want[~ok[:, None].expand(2, 2, 6)] = 7.0
    assert torch.equal(y.cpu(), want)


def steps(rot, base, scaling, factor, original, low, high):
    inv = np.float64(base) ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "linear":
        return inv / factor
    if scaling == "ntk":
        return (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "by_parts":
        keep = np.clip((original * inv / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        return inv * (keep + (1.0 - keep) / factor)
    return inv


@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
@pytest.mark.parametrize("positions", [1, 1000, 200001])
def test_tables(positions, scaling, rot):
    kw = dict(base=10000.0, scaling=scaling, factor=7.5, original=2048, low_turns=2.0, high_turns=20.0, amplitude=1.2)
    cos, sin = rope_tables(positions, rot, **kw)
    sync_status()
    inv = steps(rot, 10000.0, scaling, 7.5, 2048, 2.0, 20.0)
    rows = np.unique(np.concatenate([np.arange(min(positions, 300)), np.random.default_rng(rot).integers(0, positions, 700),
                                     [positions - 1]]))
    a = rows[:, None].astype(np.float64) * inv
    tol = float(np.float32(1.2)) * (2.5e-8 + 3 * 2.0 ** -24 + 2.0 ** -50 * rows[:, None])
    for got, want in ((cos, np.cos(a)), (sin, np.sin(a))):
        err = np.abs(got.cpu().double().numpy()[rows] - float(np.float32(1.2)) * want)
        assert (err <= tol).all(), float((err / tol).max())
    assert (cos[0] == np.float32(1.2)).all() and (sin[0] == 0).all()
    # into given tensors: the same bits
    c2, s2 = torch.zeros_like(cos), torch.zeros_like(sin)
    rope_tables(positions, rot, cos=c2, sin=s2, **kw)
    assert torch.equal(c2, cos) and torch.equal(s2, sin)


def test_autograd_captured_and_replayed_and_only_once():
    """Forward and backward captured on one stream and replayed over other
    values; a second derivative is refused, not zero."""
    B, H, L, d = 2, 3, 40, 64
    g = synth.generator(6)
    cos, sin = (t.to(DEV) for t in host_tables(L, d))
    q, k, dy, dz = (torch.zeros((B, H, L, d), device=DEV, dtype=torch.bfloat16) for _ in range(4))
    q.requires_grad_()
    k.requires_grad_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step():
        return torch.autograd.grad(rope(q, k, cos, sin, rope_interleaved=True), (q, k), (dy, dz))

    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        dq, dk = step()
    values = [synth.randn_bf16((B, H, L, d), g) for _ in range(2)]
    dy.copy_(values[0])
    dz.copy_(values[1])
    graph.replay()
    sync_status()
    at = torch.arange(L).expand(B, L)
    for got, x in zip((dq, dk), values):
        assert torch.equal(got.cpu(), turned(x, cos.cpu(), sin.cpu(), at, True, -1.0))
    y, _ = rope(q, k, cos, sin)
    first, = torch.autograd.grad((y * y).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        first.sum().backward()
