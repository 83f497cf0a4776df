"""Gradients that autograd hands over as slices of larger ones: contiguous, but at an
address that is no multiple of 16 bytes, which the kernels' wide loads need."""
import numpy as np
import pytest
import torch

from flashattention_attn_fwd_gb300 import api, attention, diff_attention, rope, rotary, sync_status, synth

DEV = "cuda"


def _slice(shape, at=3):
    """A contiguous bf16 tensor that starts `at` elements into its storage."""
    n = int(np.prod(shape))
    return torch.arange(n + 8, dtype=torch.float32).bfloat16()[at:at + n].view(shape)


@pytest.mark.parametrize("make", [lambda t: api._aligned(t), lambda t: rotary._dense(t)], ids=["attention", "rope"])
def test_a_contiguous_slice_at_an_odd_address_is_moved(make):
    t = _slice((2, 3, 4, 64))
    assert t.is_contiguous() and t.data_ptr() % 16
    got = make(t)
    assert got.data_ptr() % 16 == 0 and got.is_contiguous() and torch.equal(got, t)
    whole = t.clone()
    assert make(whole) is whole
    turned = whole.transpose(1, 2)
    got = make(turned)
    assert got.data_ptr() % 16 == 0 and torch.equal(got, turned)


def test_rope_keeps_strided_gradients_and_copies_expanded_ones():
    whole = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    assert rotary._dense(None) is None
    turned = whole.transpose(1, 2)
    assert rotary._dense(turned) is turned
    wide = torch.zeros((2, 3, 4, 68), dtype=torch.bfloat16)[..., :64]  # strides that are no multiples of 8
    for t in (wide, torch.zeros((), dtype=torch.bfloat16).expand(2, 3, 4, 64)):
        got = rotary._dense(t)
        assert got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, t)


def _grads(call, inputs, gradient, offset):
    """Gradients of `inputs` when the outputs' gradients arrive `offset` elements into
    one flat gradient."""
    leaves = [t.detach().clone().requires_grad_() for t in inputs]
    outs = call(*leaves)
    outs = outs if isinstance(outs, tuple) else (outs,)
    seen = []
    for o in outs:
        o.register_hook(lambda g: seen.append(g.data_ptr() % 16))
    head = torch.zeros(offset, device=DEV, dtype=torch.bfloat16)
    flat = torch.cat([head, *(o.reshape(-1) for o in outs)])
    flat.backward(torch.cat([head, gradient[:flat.numel() - offset]]))
    sync_status()
    return [t.grad for t in leaves], seen


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["rope", "attention", "diff"])
def test_backward_through_a_concatenation(what):
    """The same bits whether the gradient arrives aligned or not."""
    g = synth.generator(1)
    B, H, L, d = 1, 2, 80, 64
    if what == "diff":
        inputs = [t.to(DEV) for t in synth.diff_inputs(B, H, L, seed=2)]
        call, exact = lambda *a: diff_attention(*a, 0.5), (1, 3, 4)  # (dq1, dq2: sums in no fixed order)
    else:
        inputs = [synth.randn_bf16((B, H, L, d), g).to(DEV) for _ in range(2 if what == "rope" else 3)]
        a = torch.arange(L, device=DEV)[:, None] * 100.0 ** (-torch.arange(d // 2, device=DEV) * 2.0 / d)
        if what == "rope":
            call, exact = lambda q, k: rope(q, k, a.cos(), a.sin()), (0, 1)
        else:
            call, exact = lambda q, k, v: attention(q, k, v, mask="causal"), (1, 2)
    gradient = synth.randn_bf16((2 * B * H * L * 128,), g).to(DEV)
    want, _ = _grads(call, inputs, gradient, 0)
    got, seen = _grads(call, inputs, gradient, 3)
    assert any(seen)
    for i, (x, y) in enumerate(zip(got, want)):
        if i in exact:
            assert torch.equal(x, y), i
        else:
            assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max(), i
