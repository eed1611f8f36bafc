"""Rotary positions: queries and keys turned by their tokens' positions, forward and
backward, in one launch for both.

    inv_freq, scale = rotary_frequencies(128, device="cuda")
    q, k = apply_rotary(q, k, inv_freq=inv_freq, scale=scale)        # positions 0 .. N-1

    # video tokens: 128 = 44 + 42 + 42 rotated elements for time, height, width
    inv_freq, axes = axial_frequencies(128, device="cuda")
    q, k = apply_rotary(q, k, inv_freq=inv_freq, axes=axes,
                        positions=grid_positions(21, 30, 52, device="cuda"))

q and k are [B, H, N, d] with any strides over a contiguous last dimension; the
results are contiguous, as `sparse_attention` takes them, so the view
`x.view(B, N, H, d).transpose(1, 2)` of a projection needs no copy of its own. The
gradients come back in the order of q's and k's own strides.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import binding as b

_DTYPES = {torch.bfloat16: b.DTYPE_BF16, torch.float32: b.DTYPE_F32, torch.float16: b.DTYPE_F16}
_LAYOUTS = {"interleaved": b.ROTARY_INTERLEAVED, "half": b.ROTARY_HALF}


# ---- frequencies and positions --------------------------------------------------
def rotary_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cpu"):
    """(inv_freq fp64 [rotary_dim / 2], scale) of one position axis: inv_freq[p] =
    theta^(-2p / rotary_dim), stretched for contexts `factor` times as long:

    * None      as it is (factor has to be 1)
    * "linear"  every frequency divided by the factor
    * "ntk"     the base raised to theta * factor^(rd / (rd - 2)): the slowest pair is
                divided by the factor, the fastest stays
    * "yarn"    pairs that turn more than beta_fast times over original_length stay,
                those that turn less than beta_slow times are divided by the factor, a
                linear ramp over the pair index between; scale = 0.1 ln(factor) + 1
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (theta > 0 and factor >= 1.0):
        raise ValueError("theta must be positive and factor at least 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling is None and factor != 1.0:
        raise ValueError("a factor needs a scaling")
    if scaling == "yarn" and original_length < 1:
        raise ValueError('"yarn" scaling needs original_length')
    if scaling == "yarn" and not (theta > 1 and beta_fast > beta_slow > 0):
        raise ValueError('"yarn" scaling needs theta > 1 and beta_fast > beta_slow > 0')
    if scaling == "ntk" and rotary_dim > 2:
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    p = torch.arange(rotary_dim // 2, dtype=torch.float64)
    inv_freq = theta ** (-2.0 * p / rotary_dim)
    scale = 1.0
    if scaling == "linear" or (scaling == "ntk" and rotary_dim == 2):
        inv_freq = inv_freq / factor
    elif scaling == "yarn":
        def pair_of(turns):  # the (fractional) pair that turns so many times over original_length
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(theta))

        low = max(math.floor(pair_of(beta_fast)), 0)
        high = min(math.ceil(pair_of(beta_slow)), rotary_dim // 2 - 1)
        ramp = ((p - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)  # 0: kept, 1: divided
        inv_freq = inv_freq * (1.0 - ramp) + inv_freq / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    return inv_freq.to(device), scale


def axial_frequencies(rotary_dim: int, theta: float = 10000.0, device="cpu"):
    """(inv_freq, axes) for (t, h, w) grid positions: the pairs split over the three
    axes (height and width a third each, time the rest), each with its own run of
    frequencies."""
    if rotary_dim < 6 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 6 for three axes")
    pairs = rotary_dim // 2
    axes = (pairs - 2 * (pairs // 3), pairs // 3, pairs // 3)
    return torch.cat([rotary_frequencies(2 * n, theta)[0] for n in axes]).to(device), axes


def grid_positions(t: int, h: int, w: int, device="cpu") -> torch.Tensor:
    """int64 [3, t * h * w]: the (t, h, w) position of each token, flattened t-major."""
    if min(t, h, w) < 1:
        raise ValueError("a grid has at least one cell along each axis")
    n = torch.arange(t * h * w, device=device)
    return torch.stack((n // (h * w), n // w % h, n % w))


# ---- the operator ---------------------------------------------------------------
@dataclass
class Rotary:
    """The arguments of one rotation, as `sparse_attention(..., rotary=...)` takes them."""
    inv_freq: torch.Tensor
    positions: torch.Tensor | None = None
    layout: str = "interleaved"
    axes: tuple | None = None
    scale: float = 1.0


def _spec(r: Rotary, B: int, N: int, d: int, device) -> b.spa2_rotary_spec:
    f = r.inv_freq
    if r.layout not in _LAYOUTS:
        raise ValueError(f"unknown layout {r.layout!r}: 'interleaved' or 'half'")
    if f.dtype != torch.float64 or f.dim() != 1:
        raise TypeError("inv_freq must be a float64 tensor of one dimension")
    pairs = f.numel()
    if pairs < 1 or 2 * pairs > d:
        raise ValueError(f"inv_freq has {pairs} frequencies: between 1 and d / 2 = {d // 2} are wanted")
    axes = (pairs,) if r.axes is None else tuple(r.axes)
    if not 1 <= len(axes) <= b.ROTARY_MAX_AXES or min(axes) < 0 or sum(axes) != pairs:
        raise ValueError(f"axes {axes} must be 1 to {b.ROTARY_MAX_AXES} pair counts with sum {pairs}")
    if not math.isfinite(r.scale):
        raise ValueError("scale must be finite")
    pos, stride = r.positions, (0, 0, 0)
    if pos is None:
        if len(axes) != 1:
            raise ValueError("more than one axis needs positions")
    else:
        if pos.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64")
        want = (N,) if len(axes) == 1 else (len(axes), N)
        if tuple(pos.shape) == want:
            batch = 0
        elif tuple(pos.shape) == (B, *want):
            batch = pos.stride(0)
        else:
            raise ValueError(f"positions have shape {tuple(pos.shape)}: {want} or {(B, *want)} is wanted")
        stride = (batch, pos.stride(-2) if len(axes) > 1 else 0, pos.stride(-1))
    if f.device != device or (pos is not None and pos.device != device):
        raise ValueError("inv_freq and positions must be on the device of q")
    if f.stride(0) != 1:
        f = f.contiguous()
    s = b.spa2_rotary_spec()
    s.positions = None if pos is None else pos.data_ptr()
    s.position_bytes = 8 if pos is None else pos.element_size()
    s.position_stride[:] = stride
    s.axes = len(axes)
    s.pairs[:len(axes)] = axes
    s.inv_freq, s.rotary_dim, s.layout, s.scale = f.data_ptr(), 2 * pairs, _LAYOUTS[r.layout], r.scale
    s.keep = f  # the call below reads it on the current stream
    return s


def _check_inputs(xs):
    q = xs[0]
    if any(x.dtype not in _DTYPES for x in xs):
        raise TypeError("apply_rotary expects bf16, fp16 or fp32 tensors")
    if any(x.dtype != q.dtype for x in xs):
        raise TypeError("q and k must have one dtype")
    if any(x.dim() != 4 for x in xs):
        raise ValueError("apply_rotary expects [B, H, N, d] tensors")
    if any(x.device != q.device or x.device.type != "cuda" for x in xs):
        raise ValueError("apply_rotary expects tensors on one CUDA device")
    if any((x.shape[0], x.shape[2], x.shape[3]) != (q.shape[0], q.shape[2], q.shape[3]) for x in xs):
        raise ValueError("q and k must agree in batch, length and head width")


def _turn(xs, outs, r: Rotary, inverse: bool):
    """outs[i] <- xs[i] turned; every tensor [B, H, N, d] with a contiguous last dimension."""
    B, _, N, d = xs[0].shape
    spec = _spec(r, B, N, d, xs[0].device)
    pairs = [(x, y) for x, y in zip(xs, outs) if x.numel()]
    if not pairs:
        return
    t = (b.spa2_rotary_tensor * len(pairs))()
    for e, (x, y) in zip(t, pairs):
        e.x, e.y, e.heads = x.data_ptr(), y.data_ptr(), x.shape[1]
        e.x_stride[:], e.y_stride[:] = x.stride()[:3], y.stride()[:3]
    with b.on_device(xs[0].device):
        b._check(b.spa2_rotary(t, B, N, d, _DTYPES[xs[0].dtype], spec, inverse, b._stream(torch)), "spa2_rotary")


def _rows(x):
    return x if x.stride(-1) == 1 or x.shape[-1] == 1 else x.contiguous()


class RotaryFunction(torch.autograd.Function):
    """(q, k) turned by r; the backward pass is the same map with the angle negated."""

    @staticmethod
    def forward(ctx, r: Rotary, inverse: bool, strides, *xs):
        ctx.save_for_backward(r.inv_freq, r.positions)  # so that a change in between is noticed
        ctx.spec, ctx.inverse = (r.layout, r.axes, r.scale), inverse
        ctx.strides = [(x.shape, x.stride()) for x in xs]
        ctx.set_materialize_grads(False)
        xs = [_rows(x) for x in xs]
        outs = [torch.empty(x.shape, dtype=x.dtype, device=x.device) if st is None else
                torch.empty_strided(*st, dtype=x.dtype, device=x.device) for x, st in zip(xs, strides)]
        _turn(xs, outs, r, inverse)
        return tuple(outs)

    @staticmethod
    def backward(ctx, *grads):
        at = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[3 + i]]
        out = [None] * len(grads)
        if at:
            turned = RotaryFunction.apply(Rotary(*ctx.saved_tensors, *ctx.spec), not ctx.inverse, [_dense(*ctx.strides[i]) for i in at],
                                          *(grads[i] for i in at))
            for i, g in zip(at, turned):
                out[i] = g
        return (None, None, None, *out)


def _dense(shape, stride):
    """(shape, strides without gaps in the order of `stride`), None (contiguous) where that has broadcast dimensions
    or the last one is not innermost."""
    if stride[-1] != 1 and shape[-1] != 1 or any(st == 0 and size > 1 for st, size in zip(stride, shape)):
        return None
    out, n = list(stride), 1
    for i in sorted(range(len(shape)), key=lambda i: (stride[i], -i)):
        if shape[i] > 1:
            out[i] = n
            n *= shape[i]
    return shape, out


def apply_rotary(q, k=None, *, inv_freq, positions=None, layout: str = "interleaved", axes=None, scale: float = 1.0):
    """q (and k) [B, H, N, d] turned by their positions; differentiable in q and k.

    inv_freq   fp64 [rotary_dim / 2], radians per position; elements from rotary_dim on
               are passed through
    positions  int32 or int64 [N] or [B, N] (one axis), [axes, N] or [B, axes, N]
               (several); None: 0 .. N-1. Any values; negative ones turn backwards.
    layout     "interleaved": pair p is elements 2p and 2p + 1; "half": p and
               p + rotary_dim / 2
    axes       pairs per position axis, e.g. (22, 21, 21); None: one axis
    scale      factor on the rotated elements (not on the ones passed through)

    q and k are bf16, fp16 or fp32, of one dtype; their head counts may differ. Returns
    contiguous tensors: q' alone, or (q', k').
    """
    r = Rotary(inv_freq, positions, layout, axes, float(scale))
    xs = (q,) if k is None else (q, k)
    _check_inputs(xs)
    out = RotaryFunction.apply(r, False, [None] * len(xs), *xs)
    return out[0] if k is None else out
