"""Python binding of the rotary positions (include/flattn.h): rotation of queries
and keys with its gradient, and the tables that it and ``kv_append`` read.  As in
``api`` only arguments are marshalled here; the library's kernels do the work.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .api import _aligned, _empty_on, _need, _raw_stream, _stream_ptr
from ._lib import ROPE_SCALINGS, ROPE_ZERO_K, ROPE_ZERO_Q

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


_Tensor = torch.Tensor
_device_index = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_NONE = (0, 0, 0)


def _check(t, name: str, ndim: int, dtype, index: int) -> None:
    """`t` is a tensor of this rank and type on CUDA device `index`."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.dim() != ndim or t.get_device() != index:
        _need(t, name, ndim, dtype)
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _rows(t, name, shape, index):
    """Checks a [B, H, L, d] bf16 tensor; returns its (b, h, l) strides (those of
    axes of length 1 are never used to step)."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.get_device() != index or t.shape != shape:
        _check(t, name, 4, _BF16, index)
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    sb, sh, sl, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{name} must have a contiguous head dimension")
    B, H, L, d = shape
    # (all zeros would read as contiguous)
    if (B > 1 and sb == 0) or (H > 1 and sh == 0) or (L > 1 and sl == 0):
        raise ValueError(f"{name} must not be expanded")
    return sb if B > 1 else H * L * d, sh if H > 1 else L * d, sl if L > 1 else d


def _rotate(call, names, q, k, rope_cos, rope_sin, positions, rope_interleaved, q_out, k_out, stream):
    _need(q, names[0], 4)
    shape = q.shape
    B, Hq, L, d = shape
    index = q.get_device()
    if _device_index() != index:
        raise ValueError(f"{names[0]} is on cuda:{index}, the current device is cuda:{_device_index()}")
    qs = _rows(q, names[0], shape, index)
    _check(rope_cos, "rope_cos", 2, _F32, index)
    _check(rope_sin, "rope_sin", 2, _F32, index)
    tables = rope_cos.shape
    if rope_sin.shape != tables or not rope_cos.is_contiguous() or not rope_sin.is_contiguous():
        raise ValueError("rope_cos and rope_sin must be contiguous and of one shape")
    rows, half = tables
    device = q.device
    qos = kos = ks = _NONE
    Hk = kp = kop = 0
    # rows without a position in the tables: left in tensors that are given, zeros in others
    layout = 1 if rope_interleaved else 0
    if q_out is None:
        layout |= ROPE_ZERO_Q
        q_out = _empty_on(stream, shape, _BF16, device)
    else:
        qos = _rows(q_out, names[2], shape, index)
    if k is not None:
        _check(k, names[1], 4, _BF16, index)
        kshape = k.shape
        Hk = kshape[1]
        if kshape[0] != B or kshape[2] != L or kshape[3] != d:
            raise ValueError(f"{names[1]} must be [{B}, heads, {L}, {d}], got {list(kshape)}")
        ks = _rows(k, names[1], kshape, index)
        if k_out is None:
            layout |= ROPE_ZERO_K
            k_out = _empty_on(stream, kshape, _BF16, device)
        else:
            kos = _rows(k_out, names[3], kshape, index)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError(f"{names[3]} needs {names[1]}")
    pos = pos_stride = 0
    if positions is not None:
        n = positions.dim() if isinstance(positions, _Tensor) else 2
        _check(positions, "positions", n, _I32, index)
        if positions.shape != ((B, L) if n == 2 else (L,)):
            raise ValueError(f"positions must be [{B}, {L}] or [{L}], got {list(positions.shape)}")
        steps = positions.stride()
        if L > 1 and steps[-1] != 1:
            raise ValueError("positions must have contiguous rows")
        pos = positions.data_ptr()
        pos_stride = steps[0] if n == 2 and B > 1 else 0
    desc = _lib.ROPE_PACK(B, L, Hq, Hk, d, rows, 2 * half, layout, rope_cos.data_ptr(),
                          rope_sin.data_ptr(), pos, pos_stride, *qs, *ks, *qos, *kos,
                          _raw_stream(index) if stream is None else _stream_ptr(stream))
    L_ = _lib.lib()
    st = (L_.fl_rope_bwd if call == "fl_rope_bwd" else L_.fl_rope_fwd)(q.data_ptr(), kp, q_out.data_ptr(), kop, desc)
    if st:
        _lib.check(st, call)
    return q_out, k_out


def rope_fwd(q, k, rope_cos, rope_sin, *, positions=None, rope_interleaved: bool = False, q_out=None, k_out=None,
             stream=None):
    """fl_rope_fwd: rotate q [B, Hq, L, d] and k [B, Hk, L, d] (or None), bf16
    with any strides that are multiples of 8, by positions (int32 [B, L] or [L];
    None: row l has position l); rope_cos, rope_sin fp32 [positions, rope_dim /
    2].  Returns (q_out, k_out), contiguous when not given.  Rows whose position is
    outside the tables are reported by sync_status; given outputs keep what they
    held there, others get zeros."""
    return _rotate("fl_rope_fwd", ("q", "k", "q_out", "k_out"), q, k, rope_cos, rope_sin, positions, rope_interleaved,
                   q_out, k_out, stream)


def rope_bwd(dq_out, dk_out, rope_cos, rope_sin, *, positions=None, rope_interleaved: bool = False, dq=None, dk=None,
             stream=None):
    """fl_rope_bwd: gradients (dq, dk) of rope_fwd's q and k for those of its
    outputs, dq_out and dk_out (or None); the other arguments are the forward's."""
    return _rotate("fl_rope_bwd", ("dq_out", "dk_out", "dq", "dk"), dq_out, dk_out, rope_cos, rope_sin, positions,
                   rope_interleaved, dq, dk, stream)


def _dense(t):
    """A gradient with strides and an address that the kernel takes (an expanded one
    has zero strides, a slice of a larger one may start anywhere)."""
    if t is None or (t.stride(3) == 1 and all(s > 0 and s % 8 == 0 for s in t.stride()[:3]) and t.data_ptr() % 16 == 0):
        return t
    return _aligned(t)


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, rope_cos, rope_sin, positions, interleaved):
        ctx.save_for_backward(rope_cos, rope_sin, positions)
        ctx.interleaved = interleaved
        return rope_fwd(q, k, rope_cos, rope_sin, positions=positions, rope_interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        rope_cos, rope_sin, positions = ctx.saved_tensors
        dq, dk = rope_bwd(_dense(dq_out), _dense(dk_out), rope_cos, rope_sin, positions=positions,
                          rope_interleaved=ctx.interleaved)
        return dq, dk, None, None, None, None


def rope(q, k, rope_cos, rope_sin, *, positions=None, rope_interleaved: bool = False):
    """Differentiable rotation of q and k (once; the tables have no gradient):
    rope_fwd in the forward, rope_bwd in the backward.  Returns contiguous (q, k)
    as ``attention`` takes them.  Rows whose position is outside the tables (reported
    by sync_status) come out as zeros, and so do their gradients."""
    if rope_cos.requires_grad or rope_sin.requires_grad:
        raise ValueError("rope_cos and rope_sin have no gradient: detach them")
    return _Rope.apply(q, k, rope_cos, rope_sin, positions, rope_interleaved)


def rope_tables(positions: int, rope_dim: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                original: int = 0, low_turns: float = 1.0, high_turns: float = 32.0, amplitude: float = 1.0, cos=None,
                sin=None, device="cuda", stream=None):
    """fl_rope_tables: (cos, sin) fp32 [positions, rope_dim / 2] of position times
    base^(-2i / rope_dim), times amplitude.  For contexts longer than the model
    was trained on, scaling "linear" (positions / factor), "ntk" (a larger base)
    or "by_parts" (pairs that turn at least high_turns times in the ``original``
    positions stay, those below low_turns are interpolated by factor)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}")
    positions, rope_dim = int(positions), int(rope_dim)
    shape = (positions, rope_dim // 2)
    if cos is None:
        cos = _empty_on(stream, shape, _F32, torch.device(device) if sin is None else sin.device)
    if sin is None:
        sin = _empty_on(stream, shape, _F32, cos.device)
    _need(cos, "cos", 2, _F32)
    index = cos.get_device()
    _check(sin, "sin", 2, _F32, index)
    if _device_index() != index:
        raise ValueError(f"cos is on cuda:{index}, the current device is cuda:{_device_index()}")
    if cos.shape != shape or sin.shape != shape or not cos.is_contiguous() or not sin.is_contiguous():
        raise ValueError(f"cos and sin must be contiguous {list(shape)}, got {list(cos.shape)} and {list(sin.shape)}")
    spec = _lib.SCALING_PACK(base, factor, low_turns, high_turns, ROPE_SCALINGS[scaling], original, amplitude, 0)
    st = _lib.lib().fl_rope_tables(cos.data_ptr(), sin.data_ptr(), positions, rope_dim, spec,
                                   _raw_stream(index) if stream is None else _stream_ptr(stream))
    if st:
        _lib.check(st, "fl_rope_tables")
    return cos, sin
