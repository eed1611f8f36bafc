"""Rotary positions on the GPU against the formula in float64.

Tolerance. With (a, b) a pair, the kernel computes scale * (a cos - b sin, a sin + b
cos) in fp32 and rounds once. Its cos and sin are off by at most 5e-7: the angle,
reduced to [-1/2, 1/2] turns in fp64, is rounded to fp32 (2^-25 half turns = 9.4e-8
rad), the function is good to 2 ulp (2.4e-7), the product with the scale adds 2^-24,
and for |position| <= 131071 the fp64 product adds less than 1e-9. Each of the two
products and the sum rounds by 2^-24 relative. So before the last rounding the
result is within 1e-6 * scale * (|a| + |b|), and the element type adds half a step,
eps / 2 of the value (for fp16 at least half a subnormal step, 2^-25)."""

import math

import pytest
import torch

from trainable_block_sparse_pooled_b200.rotary import apply_rotary, axial_frequencies, grid_positions, rotary_frequencies

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def turned(x, angle, layout, scale, sign=1.0):
    """x [B, H, N, d] in float64 turned by angle [B or 1, N, rd / 2], and the error bound before rounding."""
    x = x.detach().double()
    rd = 2 * angle.shape[-1]
    c, s = scale * torch.cos(angle)[:, None], scale * sign * torch.sin(angle)[:, None]
    i = torch.arange(0, rd, 2, device=x.device) if layout == "interleaved" else torch.arange(rd // 2, device=x.device)
    j = i + (1 if layout == "interleaved" else rd // 2)
    y, bound = x.clone(), torch.zeros_like(x)
    a, w = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - w * s, a * s + w * c
    bound[..., i] = bound[..., j] = 1e-6 * scale * (a.abs() + w.abs())
    return y, bound


def angles(positions, inv_freq, axes):
    p = positions.double()
    if len(axes) == 1:
        return (p if p.dim() == 2 else p[None])[..., None] * inv_freq
    p = p if p.dim() == 3 else p[None]
    axis = torch.tensor([a for a, n in enumerate(axes) for _ in range(n)], device=p.device, dtype=torch.long)
    return p[:, axis].transpose(1, 2) * inv_freq


def assert_turned(got, x, angle, layout, scale, sign=1.0):
    want, bound = turned(x, angle, layout, scale, sign)
    assert got.dtype == x.dtype and got.shape == x.shape
    eps = torch.finfo(x.dtype).eps
    tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}[x.dtype]
    err = (got.double() - want).abs() - (bound + eps / 2 * (want.abs() + bound) + tiny)
    assert err.max() <= 0, f"worst excess {err.max():.3e}"
    rd = 2 * angle.shape[-1]
    assert torch.equal(got[..., rd:], x[..., rd:])


CASES = [
    # B, N, Hq, Hk, d, rd, layout, dtype, axes, positions, order
    (1, 1, 1, 1, 64, 64, "interleaved", BF16, 1, "none", "bhnd"),
    (8, 1, 32, 8, 128, 128, "half", BF16, 1, "far", "bnhd"),
    (2, 130, 3, 3, 128, 128, "interleaved", BF16, 3, "grid", "bnhd"),
    (2, 130, 3, 1, 128, 64, "half", BF16, 2, "batch", "bnhd"),
    (3, 77, 5, 2, 80, 40, "half", F16, 1, "batch", "bnhd"),       # pairs 20 apart: no 16-byte units
    (3, 77, 5, 2, 80, 40, "interleaved", F16, 1, "i32", "bhnd"),
    (1, 257, 2, 7, 96, 48, "half", F32, 4, "batch", "bnhd"),
    (1, 33, 4, 4, 256, 256, "interleaved", F32, 1, "negative", "bnhd"),
    (2, 19, 2, 2, 7, 2, "interleaved", BF16, 1, "none", "bhnd"),  # odd width, one pair
    (2, 19, 2, 2, 7, 6, "half", F32, 1, "far", "bnhd"),
    (1, 5, 1, 1, 1024, 1022, "half", BF16, 1, "none", "bnhd"),
    (1, 1000, 12, 12, 128, 128, "interleaved", BF16, 3, "grid", "bnhd"),
]


@pytest.mark.parametrize("B,N,Hq,Hk,d,rd,layout,dtype,axes,kind,order", CASES)
def test_forward_and_gradients(B, N, Hq, Hk, d, rd, layout, dtype, axes, kind, order):
    g = torch.Generator(device="cuda").manual_seed(N * 1000 + d)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    make = lambda H: rand(B, N, H, d).transpose(1, 2) if order == "bnhd" else rand(B, H, N, d)  # noqa: E731
    pairs = rd // 2
    inv_freq = rotary_frequencies(rd, device="cuda")[0]
    split = {1: (pairs,), 2: (pairs - 5, 5), 3: (pairs - 2 * (pairs // 3), pairs // 3, pairs // 3),
             4: (3, 0, pairs - 4, 1)}[axes]
    if kind == "grid":
        pos = grid_positions(-(-N // 35), 5, 7, device="cuda")[:, :N]   # a slice: strides of its own
        split, inv_freq = axial_frequencies(rd, device="cuda")[::-1]
    elif kind == "batch":
        pos = torch.randint(0, 5000, (B, N) if axes == 1 else (B, axes, N), generator=g, device="cuda")
    else:
        pos = {"none": torch.arange(N, device="cuda"), "far": torch.arange(N, device="cuda") + 131071 - N,
               "i32": torch.arange(N, device="cuda", dtype=torch.int32) * 3,
               "negative": torch.arange(N, device="cuda") - 500}[kind]
    scale = 1.0 if kind != "far" else 1.1386294361119891
    q, k = make(Hq).requires_grad_(), make(Hk).requires_grad_()
    yq, yk = apply_rotary(q, k, inv_freq=inv_freq, positions=None if kind == "none" else pos, layout=layout,
                          axes=None if axes == 1 else split, scale=scale)
    angle = angles(pos, inv_freq, split)
    for y, x in ((yq, q), (yk, k)):
        assert y.is_contiguous()
        assert_turned(y.detach(), x.detach(), angle, layout, scale)
    dq, dk = rand(B, Hq, N, d), make(Hk)   # one gradient contiguous, the other as the inputs lie
    gq, gk = torch.autograd.grad((yq, yk), (q, k), (dq, dk))
    for y, x, leaf in ((gq, dq, q), (gk, dk, k)):
        assert_turned(y, x, angle, layout, scale, sign=-1.0)
        assert y.stride() == leaf.stride()


def test_gradient_against_differences():
    """The map is linear, so <g, apply(x + v) - apply(x)> = <grad(g), v>. In fp32, each
    side of the identity is a sum over elements; every element of apply is within
    1e-6 (|a| + |b|) + 2^-24 |y| <= 2e-6 (|a| + |b|) of its value, the rounding of x + v
    (2^-24 |x + v|) is taken out by using x + v as rounded."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, v, h = (torch.randn(1, 2, 50, 64, generator=g, device="cuda") for _ in range(3))
    f = rotary_frequencies(48, device="cuda")[0]
    xv = x + v
    leaf = x.clone().requires_grad_()
    y = apply_rotary(leaf, inv_freq=f, scale=1.25)
    (grad,) = torch.autograd.grad(y, leaf, h)
    left = (h.double() * (apply_rotary(xv, inv_freq=f, scale=1.25).double() - y.detach().double())).sum()
    right = (grad.double() * (xv.double() - x.double())).sum()
    size = lambda t: t.abs().double().sum(-1, keepdim=True)  # noqa: E731  (|a| + |b| <= the row's sum)
    bound = 1.25 * 2e-6 * ((h.abs().double() * (size(xv) + size(x))).sum() + ((xv - x).abs().double() * size(h)).sum())
    assert abs(left - right) <= bound


def test_only_what_needs_a_gradient_gets_one():
    f = rotary_frequencies(64, device="cuda")[0]
    q = torch.randn(1, 2, 9, 64, device="cuda", requires_grad=True)
    k = torch.randn(1, 1, 9, 64, device="cuda")
    yq, yk = apply_rotary(q, k, inv_freq=f)
    yq.sum().backward()
    want, = torch.autograd.grad(apply_rotary(q, inv_freq=f).sum(), q)
    assert torch.equal(q.grad, want) and k.grad is None
    # only one of two results used; and nothing wanted at all
    k.requires_grad_()
    yq, yk = apply_rotary(q, k, inv_freq=f)
    gq, gk = torch.autograd.grad(yk.sum(), (q, k), allow_unused=True)
    assert gq is None and gk is not None
    with torch.no_grad():
        assert not apply_rotary(q, inv_freq=f).requires_grad


def test_second_derivative_and_broadcast_input():
    """grad of grad turns forward again; a broadcast batch sums its gradients."""
    f = rotary_frequencies(64, device="cuda")[0]
    x = torch.randn(1, 2, 9, 64, device="cuda", requires_grad=True)
    w = torch.randn(3, 2, 9, 64, device="cuda", requires_grad=True)
    y = apply_rotary(x.expand(3, -1, -1, -1), inv_freq=f)
    (gx,) = torch.autograd.grad(y, x, w, create_graph=True)
    each = [torch.autograd.grad(apply_rotary(x, inv_freq=f), x, w[i:i + 1].detach())[0] for i in range(3)]
    assert torch.allclose(gx, sum(each), rtol=1e-6, atol=1e-6)   # sums of three in another order: 2 * 2^-24 * |sum|
    (gw,) = torch.autograd.grad(gx, w, x.detach())
    assert torch.equal(gw, apply_rotary(x.detach(), inv_freq=f).expand(3, -1, -1, -1))


def test_positions_changed_in_place_are_noticed():
    f = rotary_frequencies(64, device="cuda")[0]
    x = torch.randn(1, 1, 4, 64, device="cuda", requires_grad=True)
    pos = torch.arange(4, device="cuda")
    y = apply_rotary(x, inv_freq=f, positions=pos)
    pos += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()


def _layouts(g):
    """Inputs [2, 3, 21, 64] bf16 in unusual places, by name."""
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    yield "slice of a fused projection", r(2, 21, 3, 3, 64)[:, :, 1].transpose(1, 2)
    yield "slice along the width", r(2, 3, 21, 80)[..., 5:69]
    yield "odd token stride", r(2, 3, 21, 67)[..., :64]
    yield "odd storage offset", r(2 * 3 * 21 * 64 + 1)[1:].view(2, 3, 21, 64)
    yield "8-byte offset", r(2 * 3 * 21 * 64 + 4)[4:].view(2, 3, 21, 64)
    yield "tokens last", r(2, 3, 64, 21).transpose(2, 3)
    yield "broadcast batch", r(1, 3, 21, 64).expand(2, -1, -1, -1)
    yield "broadcast heads", r(2, 1, 21, 64).expand(-1, 3, -1, -1)
    yield "reversed order", r(21, 3, 2, 64).permute(2, 1, 0, 3)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_strides_and_alignments(layout):
    g = torch.Generator(device="cuda").manual_seed(5)
    f = rotary_frequencies(32, device="cuda")[0]
    for name, x in _layouts(g):
        want = apply_rotary(x.contiguous().clone(), inv_freq=f, layout=layout)
        leaf = x.detach().requires_grad_()
        y = apply_rotary(leaf, inv_freq=f, layout=layout)
        assert torch.equal(y, want), name
        assert_turned(y.detach(), x, angles(torch.arange(21, device="cuda"), f, (16,)), layout, 1.0)
        h = torch.randn(2, 3, 21, 64, generator=g, device="cuda").to(BF16)
        (grad,) = torch.autograd.grad(y, leaf, h)
        assert_turned(grad, h, angles(torch.arange(21, device="cuda"), f, (16,)), layout, 1.0, sign=-1.0)


def test_infinities_and_nan_stay_in_their_pair():
    f = rotary_frequencies(64, device="cuda")[0]
    for layout, other in (("interleaved", 11), ("half", 42)):
        x = torch.randn(1, 2, 40, 96, device="cuda", dtype=F32).to(BF16)
        y = apply_rotary(x, inv_freq=f, layout=layout)
        bad = x.clone()
        bad[0, 1, 7, 10] = math.nan
        bad[0, 0, 3, 10] = math.inf
        bad[0, 0, 9, 90] = -math.inf      # a copied element
        z = apply_rotary(bad, inv_freq=f, layout=layout)
        assert torch.isnan(z[0, 1, 7, [10, other]]).all() and not torch.isfinite(z[0, 0, 3, [10, other]]).any()
        assert z[0, 0, 9, 90] == -math.inf
        keep = torch.ones_like(x, dtype=torch.bool)
        keep[0, 1, 7, [10, other]] = keep[0, 0, 3, [10, other]] = False
        keep[0, 0, 9, 90] = False
        assert torch.equal(z[keep], y[keep])


def test_far_positions_and_large_frequencies():
    """Positions to 2^31 and frequencies above a turn per position: the fp64 product of
    position and turns is off by 3 roundings of 2^-53, up to 2^31 * f / 2 pi * 3 *
    2^-53 turns = 2^31 f * 3.4e-16 rad; for f <= 4 that is 3e-6."""
    f = torch.tensor([4.0, 3.7, 1.0, 1e-3, 7e-5, -0.3], dtype=torch.float64, device="cuda")
    pos = torch.tensor([0, 1, -1, 131072, 2 ** 31 - 1, -2 ** 31], device="cuda")
    x = torch.randn(1, 1, 6, 12, device="cuda")
    y = apply_rotary(x, inv_freq=f, positions=pos)
    # exact angles: whole turns taken out in integers of 2^-200 turns
    import fractions
    pi = fractions.Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    ang = [[float((p * fractions.Fraction(w)) % (2 * pi)) for w in f.tolist()] for p in pos.tolist()]
    want, bound = turned(x, torch.tensor(ang, dtype=torch.float64, device="cuda")[None], "interleaved", 1.0)
    assert ((y.double() - want).abs() <= 4.5 * bound + 2.0 ** -24 * want.abs()).all()


def test_more_than_2_31_elements():
    """Offsets beyond 32 bits, in the input's and the output's strides."""
    B, H, N, d = 1, 130, 131072, 128
    x = torch.empty(B, N, H, d, dtype=BF16, device="cuda")
    x[:, -300:] = torch.randn(300, H, d, device="cuda").to(BF16)
    x[:, :300] = torch.randn(300, H, d, device="cuda").to(BF16)
    q = x.transpose(1, 2)
    f = rotary_frequencies(d, device="cuda")[0]
    y = apply_rotary(q, inv_freq=f)
    pos = torch.arange(N, device="cuda")
    for part in (slice(0, 300), slice(N - 300, N)):
        assert_turned(y[:, :, part], q[:, :, part], angles(pos[part], f, (64,)), "interleaved", 1.0)


def test_more_tokens_than_a_grid_axis():
    """B * N beyond 65535 * 16 tokens of a narrow head, and many heads."""
    f = rotary_frequencies(2, device="cuda")[0]
    x = torch.randn(2, 1, 1200000, 2, device="cuda")
    pos = torch.arange(1200000, device="cuda") % 1000
    assert_turned(apply_rotary(x, inv_freq=f, positions=pos), x, angles(pos, f, (1,)), "interleaved", 1.0)
    x = torch.randn(1, 65535, 2, 8, device="cuda")
    f = rotary_frequencies(8, device="cuda")[0]
    assert_turned(apply_rotary(x, inv_freq=f), x, angles(torch.arange(2, device="cuda"), f, (4,)), "interleaved", 1.0)


def test_empty_inputs():
    f = rotary_frequencies(64, device="cuda")[0]
    for shape in ((0, 2, 5, 64), (1, 0, 5, 64), (1, 2, 0, 64)):
        q = torch.zeros(shape, device="cuda", requires_grad=True)
        y = apply_rotary(q, inv_freq=f)
        assert y.shape == shape
        y.sum().backward()
    yq, yk = apply_rotary(torch.ones(1, 2, 5, 64, device="cuda"), torch.zeros(1, 0, 5, 64, device="cuda"), inv_freq=f)
    assert yk.numel() == 0 and torch.equal(yq, apply_rotary(torch.ones(1, 2, 5, 64, device="cuda"), inv_freq=f))


def test_width_beyond_the_supported_set_is_refused():
    from trainable_block_sparse_pooled_b200 import binding as b
    with pytest.raises(b.Spa2Error) as e:
        apply_rotary(torch.zeros(1, 1, 2, 1028, device="cuda"), inv_freq=rotary_frequencies(64, device="cuda")[0])
    assert e.value.code == b.ERR_UNSUPPORTED


def test_side_stream_and_captured_replays():
    """A call on a side stream; a captured forward and backward replayed on new inputs
    and new positions, on another stream than it was captured on."""
    f = rotary_frequencies(128, device="cuda")[0]
    q = torch.randn(2, 4, 100, 128, device="cuda").to(BF16)
    h = torch.randn(2, 4, 100, 128, device="cuda").to(BF16)
    pos = torch.arange(100, device="cuda")

    def step(x, p, grad):
        x = x.detach().requires_grad_()
        y = apply_rotary(x, inv_freq=f, positions=p)
        return y.detach(), torch.autograd.grad(y, x, grad)[0]

    want = step(q, pos, h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(q, pos, h)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(q, pos, h)
    q.copy_(torch.randn_like(q))
    pos += 1000
    want = step(q, pos, h)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(out, want))
