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
from torch.autograd import forward_ad

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
        high = min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)  # may lie behind the last pair, rotary_dim / 2 - 1
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


def _spec(r: Rotary, B: int, N: int, d: int, device) -> tuple:
    """(spa2_rotary_spec as bytes, the tensors it points into) of r for q and k [B, H, N, d]."""
    f, pos = r.inv_freq, r.positions
    layout = _LAYOUTS.get(r.layout)
    if layout is None:
        raise ValueError(f"unknown layout {r.layout!r}: 'interleaved' or 'half'")
    if f.dtype != torch.float64 or f.dim() != 1:
        raise TypeError("inv_freq must be a float64 tensor of one dimension")
    if f.requires_grad:
        raise ValueError("inv_freq takes no gradient: detach it")
    pairs = f.shape[0]
    if pairs < 1 or 2 * pairs > d:
        raise ValueError(f"inv_freq has {pairs} frequencies: between 1 and d / 2 = {d // 2} are wanted")
    axes = (pairs,) if r.axes is None else tuple(r.axes)
    n_axes = len(axes)
    if not 1 <= n_axes <= b.ROTARY_MAX_AXES or min(axes) < 0 or sum(axes) != pairs:
        raise ValueError(f"axes {axes} must be 1 to {b.ROTARY_MAX_AXES} pair counts with sum {pairs}")
    if not math.isfinite(r.scale):
        raise ValueError("scale must be finite")
    at, size, stride = None, 8, (0, 0, 0)
    if pos is None:
        if n_axes != 1:
            raise ValueError("more than one axis needs positions")
    else:
        if pos.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64")
        want = (N,) if n_axes == 1 else (n_axes, N)
        shape = tuple(pos.shape)
        if shape != want and shape != (B, *want):
            raise ValueError(f"positions have shape {shape}: {want} or {(B, *want)} is wanted")
        if pos.device != device:
            raise ValueError("positions must be on the device of q")
        at, size, stride = b.rotary_positions(pos, n_axes)
    if f.device != device:
        raise ValueError("inv_freq must be on the device of q")
    if f.stride(0) != 1:
        f = f.contiguous()
    return b.rotary_spec(at, size, stride, axes, f.data_ptr(), 2 * pairs, layout, r.scale), f


def _turned(spec, inverse: bool, strides, xs):
    """xs turned by the spa2_rotary_spec `spec`, each in strides of its own or (None) contiguous."""
    x = xs[0]
    (B, _, N, d), dtype = x.shape, x.dtype
    fields, outs, keep = [], [], []
    for x, st in zip(xs, strides):
        xb, xh, xn, xe = x.stride()
        if xe != 1 and d != 1:
            x = x.contiguous()
            keep.append(x)
            xb, xh, xn, _ = x.stride()
        y = torch.empty_like(x, memory_format=torch.contiguous_format) if st is None else \
            torch.empty_strided(x.shape, st, dtype=dtype, device=x.device)
        outs.append(y)
        heads = x.shape[1]
        if B and heads and N:
            yb, yh, yn, _ = y.stride()
            fields += x.data_ptr(), y.data_ptr(), heads, xb, xh, xn, yb, yh, yn
    n = len(fields) // 9
    if n:
        rc = b.launch(b.lib().spa2_rotary, x.device, b.ROTARY_TENSORS[n].pack(*fields), n, B, N, d, _DTYPES[dtype], spec,
                      inverse)
        if rc != b.OK:
            raise b.Spa2Error(rc, "spa2_rotary")
    return outs


class RotaryFunction(torch.autograd.Function):
    """(q, k) turned by Rotary(inv_freq, positions, *how); the backward pass is the same map with the angle
    negated, the forward-mode derivative the same map of the tangents."""

    @staticmethod
    def forward(ctx, how: tuple, inverse: bool, strides, inv_freq, positions, *xs):
        B, _, N, d = xs[0].shape
        spec, f = _spec(Rotary(inv_freq, positions, *how), B, N, d, xs[0].device)
        ctx.save_for_backward(inv_freq, positions)  # so that a change in between is noticed
        ctx.how, ctx.spec, ctx.inverse = how, spec, inverse
        ctx.strides = [_dense(x) for x in xs]
        if forward_ad._current_level >= 0:  # for jvp, which follows at once
            ctx.save_for_forward(inv_freq, positions)
            ctx.out_strides, ctx.shapes = strides, [x.shape for x in xs]
        ctx.set_materialize_grads(False)
        return tuple(_turned(spec, inverse, strides, xs))

    @staticmethod
    def jvp(ctx, _how, _inverse, _strides, freq_tangent, _positions, *tangents):
        if freq_tangent is not None:
            raise RuntimeError("inv_freq takes no derivative: detach it")
        at = [i for i, t in enumerate(tangents) if t is not None]
        turned = iter(RotaryFunction.apply(ctx.how, ctx.inverse, [ctx.out_strides[i] for i in at], *ctx.saved_tensors,
                                           *[tangents[i] for i in at]))
        return tuple([next(turned) if t is not None else tangents[at[0]].new_zeros(shape)
                      for t, shape in zip(tangents, ctx.shapes)])

    @staticmethod
    def backward(ctx, *grads):
        wanted = ctx.needs_input_grad
        at = [i for i, g in enumerate(grads) if g is not None and wanted[5 + i]]
        out = [None] * len(grads)
        if at:
            inv_freq, positions = ctx.saved_tensors
            strides, xs = [ctx.strides[i] for i in at], [grads[i] for i in at]
            if torch.is_grad_enabled():  # the gradient will be differentiated itself
                turned = RotaryFunction.apply(ctx.how, not ctx.inverse, strides, inv_freq, positions, *xs)
            else:
                B, _, N, d = xs[0].shape
                spec, f = ctx.spec, None
                if not b.rotary_spec_points(spec, inv_freq, positions):  # copies of the saved tensors
                    spec, f = _spec(Rotary(inv_freq, positions, *ctx.how), B, N, d, xs[0].device)
                turned = _turned(spec, not ctx.inverse, strides, xs)
            for i, g in zip(at, turned):
                out[i] = g
        return (None, None, None, None, None, *out)


def _has_tangent(*xs) -> bool:
    """Whether one of xs is a dual tensor of forward-mode differentiation."""
    return forward_ad._current_level >= 0 and any([forward_ad.unpack_dual(x).tangent is not None for x in xs])


def _dense(x):
    """Strides without gaps in the order of x's, or None (contiguous) where x has broadcast dimensions or its
    last dimension is not innermost."""
    shape, stride = x.shape, x.stride()
    if x.is_contiguous():
        return stride
    if stride[-1] != 1 and shape[-1] != 1 or any(st == 0 and size > 1 for st, size in zip(stride, shape)):
        return None
    out, n = list(stride), 1
    for i in sorted(range(len(shape)), key=lambda i: (stride[i], -i)):
        if shape[i] > 1:
            out[i] = n
            n *= shape[i]
    return out


def apply_rotary(q, k=None, *, inv_freq, positions=None, layout: str = "interleaved", axes=None, scale: float = 1.0):
    """q (and k) [B, H, N, d] turned by their positions; differentiable in q and k, any number of times and in
    forward mode too.

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
    if getattr(scale, "requires_grad", False):
        raise ValueError("scale takes no gradient: give a number")
    dtype, device = q.dtype, q.device
    if dtype not in _DTYPES or k is not None and k.dtype not in _DTYPES:
        raise TypeError("apply_rotary expects bf16, fp16 or fp32 tensors")
    if k is not None and k.dtype != dtype:
        raise TypeError("q and k must have one dtype")
    if q.dim() != 4 or k is not None and k.dim() != 4:
        raise ValueError("apply_rotary expects [B, H, N, d] tensors")
    if device.type != "cuda" or k is not None and k.device != device:
        raise ValueError("apply_rotary expects tensors on one CUDA device")
    xs, wanted = (q,), q.requires_grad
    if k is not None:
        xs, wanted = (q, k), wanted or k.requires_grad
        (B, _, N, d), other = q.shape, k.shape
        if other[0] != B or other[2] != N or other[3] != d:
            raise ValueError("q and k must agree in batch, length and head width")
    if wanted and torch.is_grad_enabled() or torch.jit.is_tracing() or _has_tangent(inv_freq, *xs):
        out = RotaryFunction.apply((layout, axes, float(scale)), False, (None, None), inv_freq, positions, *xs)
    else:
        B, _, N, d = q.shape
        spec, f = _spec(Rotary(inv_freq, positions, layout, axes, float(scale)), B, N, d, device)
        out = tuple(_turned(spec, False, (None, None), xs))
    return out[0] if k is None else out
