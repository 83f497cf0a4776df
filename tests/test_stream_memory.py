"""Outputs and workspaces that a call allocates belong to the stream that its
kernels run on, whichever way that stream is named: none, a torch stream, a raw
handle, or 0, the legacy default stream (a torch stream wrapped around a null
handle is another one, out of torch's pool)."""
import contextlib

import pytest
import torch

from flashattention_attn_fwd_gb300 import api, attn_bwd, attn_fwd, synth, sync_status

DEV = "cuda"


def test_stream_zero_is_the_default_stream(monkeypatch):
    """No GPU: which stream the allocation is made under."""
    made, used = [], []

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle
            made.append(handle)

    default = object()
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)

    @contextlib.contextmanager
    def under(stream):
        used.append(stream)
        yield
    monkeypatch.setattr(torch.cuda, "stream", under)

    class Other:  # a stream object of another library
        def __init__(self, handle):
            self.cuda_stream = handle
    for stream in (0, Other(0)):
        api._empty_on(stream, (4,), torch.uint8, "cpu")
        assert used.pop() is default and not made
    for stream in (0x1230, Other(0x1230)):
        api._empty_on(stream, (4,), torch.uint8, "cpu")
        assert used.pop().cuda_stream == 0x1230 and made.pop() == 0x1230
    api._empty_on(None, (4,), torch.uint8, "cpu")
    assert not used and not made


def _owner(t):
    """The stream whose pool holds t's memory (the allocator's record)."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.gpu
def test_allocations_belong_to_the_named_stream():
    q, k, v = (t.to(DEV) for t in synth.attn_inputs(1, 2, 2, 300, 64, seed=1))
    dout = torch.ones_like(q)
    kw = dict(mask="window", window=64, sink=4)
    out, lse = attn_fwd(q, k, v, **kw)
    want = attn_bwd(q, k, v, out, dout, lse, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # the current stream is another one than the calls'
    with torch.cuda.stream(torch.cuda.Stream()):
        for stream, handle in ((0, 0), (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream)):
            out, lse = attn_fwd(q, k, v, stream=stream, **kw)
            grads = attn_bwd(q, k, v, out, dout, lse, stream=stream, **kw)
            space = api._empty_on(stream, (1 << 20,), torch.uint8, q.device)
            for t in (out, lse, *grads, space):
                assert _owner(t) == handle
            sync_status(stream)
            for a, b in zip(grads[1:], want[1:]):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_every_call_allocates_on_its_stream(monkeypatch):
    """The calls with workspaces of their own: what they allocate, a workspace that
    is let go when the call returns included, belongs to the stream they run on."""
    from flashattention_attn_fwd_gb300 import (attn_decode_fwd, diffattn_bwd, diffattn_fwd, evoformer_col_gated_attn_fwd,
                                               evoformer_gated_attn_fwd)
    seen = []
    real = api._empty_on

    def spy(*args):
        t = real(*args)
        seen.append(_owner(t))
        return t
    q, k, v, kv_len = (t.to(DEV) for t in synth.decode_inputs(2, 8, 2, 1, 4096, 64, seed=1))
    diff = [t.to(DEV) for t in synth.diff_inputs(1, 2, 256, seed=2)]
    dout = torch.ones_like(diff[4])
    row = [t.to(DEV) for t in synth.evo_inputs(1, 4, 64, 2, seed=3)]
    col = [t.to(DEV) for t in synth.evo_col_inputs(1, 64, 4, 2, seed=4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls = {
        "decode": (lambda s: attn_decode_fwd(q, k, v, kv_len, stream=s), 3),       # out, lse, workspace
        "diff": (lambda s: diffattn_fwd(*diff, 0.5, stream=s), 2),
        "diff backward": (lambda s: diffattn_bwd(*diff, dout, 0.5, stream=s), 6),  # five gradients, workspace
        "row": (lambda s: evoformer_gated_attn_fwd(*row, stream=s), 2),
        "column": (lambda s: evoformer_col_gated_attn_fwd(*col, stream=s), 2),
    }
    monkeypatch.setattr(api, "_empty_on", spy)
    for name, (call, count) in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        for stream, handle in ((side, side.cuda_stream), (0, 0)):
            with torch.cuda.stream(torch.cuda.Stream()):
                seen.clear()
                got = call(stream)
                assert seen == [handle] * count, name
                sync_status(stream)
            for i, (a, b) in enumerate(zip(got, want)):
                # (dq1 and dq2 are sums in no fixed order)
                assert torch.equal(a, b) or (name == "diff backward" and i in (0, 2)), (name, i)
