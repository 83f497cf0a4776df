"""Window with sinks, backward: the first rows of a sequence see few keys at
every length, and their gradients keep the precision that short sequences and
narrow windows have.  dQ of rows 0 .. 63 depends on the first 64 tokens alone, so
its values and bound are those of the sequence cut there (a few-keys case of
the bounds in test_gpu_sink.py); peaked rows, whose dS cancels most, are brought
about by larger queries."""
import pytest

from flashattention_attn_fwd_gb300 import attn_bwd, attn_fwd, sync_status
from tests.test_gpu_sink import _bounds, _inputs, _mods, _within

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("gain", [1.0, 3.0])
@pytest.mark.parametrize("case", [
    # (B, Hq, Hkv, L, d, dv, window, sink, score mod)
    (1, 2, 2, 513, 64, 64, 256, 4, None), (2, 3, 1, 700, 64, 64, 300, 1, None), (1, 4, 2, 1026, 128, 128, 100, 40, None),
    (1, 2, 1, 515, 32, 32, 61, 4, None), (1, 2, 2, 640, 64, 128, 64, 64, None), (1, 2, 2, 600, 64, 64, 2 ** 31 - 1, 2, 5.0),
    (1, 2, 1, 900, 128, 128, 80, 600, 30.0), (1, 4, 4, 520, 64, 64, 128, 4, "alibi"),
], ids=lambda c: "-".join(str(x) for x in c))
def test_first_rows_keep_their_precision_at_every_length(case, gain):
    B, Hq, Hkv, L, d, dv, window, sink, mod = case
    q, k, v, dout = _inputs(B, Hq, Hkv, L, d, dv, seed=L + int(gain))
    q = (q.float() * gain).bfloat16()
    gkw, okw = _mods(mod, Hq)
    a = [t.to(DEV) for t in (q, k, v, dout)]
    kw = dict(mask="window", window=window, sink=sink, **gkw)
    out, lse = attn_fwd(*a[:3], **kw)
    grads = attn_bwd(*a[:3], out, a[3], lse, **kw)
    sync_status()
    n = 64
    cut = [t[:, :, :n].contiguous() for t in (q, k, v, dout)]
    r, e = _bounds(*cut, window, sink, **okw)
    _within(grads[0][:, :, :n], r["dq"], e["dq"], "dq of the first rows")
    if mod != "alibi":  # whose bound over a long sequence says little
        r, e = _bounds(q, k, v, dout, window, sink, **okw)
        for name, g in zip(("dq", "dk", "dv"), grads):
            _within(g, r[name], e[name], name)
