"""Chunk attention, cache read, rotation and tables: memory that a call allocates belongs
to the stream that it runs on, however that is named, and indices past 32 bits."""
import pytest
import torch

from flashattention_attn_fwd_gb300 import (api, attn_paged_prefill_fwd, kv_read, paged, rope_bwd, rope_fwd, rope_tables,
                                           rotary, sync_status, synth)
from tests._paged import pool, rope_tables as host_tables, table_for
from tests.test_gpu_kv_read import expected
from tests.test_gpu_paged import DEV, dev, make_cache
from tests.test_stream_memory import _owner

pytestmark = pytest.mark.gpu


def test_every_call_allocates_on_its_stream(monkeypatch):
    seen = []

    def spy(real):
        def call(*args):
            t = real(*args)
            seen.append(_owner(t))
            return t
        return call
    for module in (paged, rotary):
        for name in ("_empty_on", "_zeros_on"):
            if hasattr(module, name):
                monkeypatch.setattr(module, name, spy(getattr(api, name)))
    page, lens, new = 32, [200, 90], [40, 7]
    parts, _, _ = pool("bf16", 12, 2, page, 64, seed=1)
    cache, table = make_cache(parts), dev(table_for(lens, page, 12, seed=2))
    n, off, T = dev(lens, torch.int32), dev([0, 40, 47], torch.int32), 50
    q = synth.randn_bf16((T, 4, 64), synth.generator(3)).to(DEV)
    x = synth.randn_bf16((1, 3, 30, 64), synth.generator(4)).to(DEV)
    cos, sin = (t.to(DEV) for t in host_tables(40, 64))
    calls = {
        "chunks": (lambda s: attn_paged_prefill_fwd(q, cache, n, table, seq_offsets=off, stream=s), 3),  # and a workspace
        "read": (lambda s: kv_read(cache, n, table, T, seq_offsets=off, stream=s), 2),
        "rotation": (lambda s: rope_fwd(x, x, cos, sin, stream=s), 2),
        "its gradient": (lambda s: rope_bwd(x, x, cos, sin, stream=s), 2),
        "tables": (lambda s: rope_tables(70, 64, stream=s), 2),
    }
    side = torch.cuda.Stream()
    for name, (call, count) in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        for stream, handle in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (0, 0)):
            with torch.cuda.stream(torch.cuda.Stream()):
                seen.clear()
                got = call(stream)
                assert seen == [handle] * count, name
                sync_status(stream)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_read_from_a_pool_past_32_bits(fmt):
    """Pages whose first element lies past 2^31 (elements, and bytes)."""
    Hkv, d, page = 2, 128, 256
    pages = 2 ** 31 // (Hkv * page * (d if fmt == "bf16" else d // 2)) + 40
    small, _, _ = pool(fmt, 6, Hkv, page, d, seed=5)
    parts = []
    for t in small:
        if t is None:
            parts.append(None)
            continue
        big = torch.empty((pages, *t.shape[1:]), device=DEV, dtype=t.dtype)
        big[-6:] = t.to(DEV)
        parts.append(big)
    lens, rows = [700, 300], [700, 11]
    table = table_for(lens, page, 6, seed=6)
    k, v = kv_read(make_cache(parts), dev(lens, torch.int32), torch.where(dev(table) < 0, -1, dev(table) + pages - 6).int(),
                   711, seq_offsets=dev([0, 700, 711], torch.int32))
    sync_status()
    ek, ev = expected(make_cache(small), lens, rows, table, 711)
    assert torch.equal(k.cpu(), ek) and torch.equal(v.cpu(), ev)


@pytest.mark.parametrize("token_major", [False, True])
def test_rotation_of_more_than_2_to_the_31_elements(token_major):
    H, L, d = 2, 2 ** 24 + 50, 64
    assert H * L * d > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(7)
    shape = (1, L, H, d) if token_major else (1, H, L, d)
    x = torch.empty(shape, device=DEV, dtype=torch.bfloat16).normal_(generator=g)
    x = x.transpose(1, 2) if token_major else x
    cos, sin = (t.to(DEV) for t in host_tables(1000, d))
    pos = (torch.arange(L, device=DEV) % 1000).int()
    y, _ = rope_fwd(x, None, cos, sin, positions=pos)
    sync_status()
    for at in (0, 2 ** 23 - 20, L - 60):  # the second's rows of head 1 begin past 2^30, the last's past 2^31
        part, _ = rope_fwd(x[:, :, at:at + 60].contiguous(), None, cos, sin, positions=pos[at:at + 60])
        assert torch.equal(y[:, :, at:at + 60], part)
    dx, _ = rope_bwd(y, None, cos, sin, positions=pos, dq=torch.empty_like(x))
    part, _ = rope_bwd(y[:, :, -60:].contiguous(), None, cos, sin, positions=pos[-60:])
    sync_status()
    assert torch.equal(dx[:, :, -60:], part)
