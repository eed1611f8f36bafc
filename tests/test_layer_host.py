"""Rotary positions and 8-bit checkpoints without a GPU: frequencies and positions
against their formulas, and every refusal before anything is launched."""

import ctypes
import math

import pytest
import torch

from trainable_block_sparse_pooled_b200 import autograd, binding as b, build, checkpoint, rotary


@pytest.fixture(scope="module", autouse=True)
def L():
    build.build()
    return b.lib()


# ---- frequencies and positions -----------------------------------------------------
def test_plain_and_linear_frequencies():
    f, s = rotary.rotary_frequencies(8, theta=10000.0)
    assert f.dtype == torch.float64 and s == 1.0
    assert f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    g, s = rotary.rotary_frequencies(8, scaling="linear", factor=4.0)
    assert torch.equal(g, f / 4) and s == 1.0


def test_ntk_keeps_the_fastest_and_divides_the_slowest_pair():
    f, _ = rotary.rotary_frequencies(64)
    g, s = rotary.rotary_frequencies(64, scaling="ntk", factor=8.0)
    assert g[0] == f[0] and s == 1.0
    assert g[-1].item() == pytest.approx(f[-1].item() / 8, rel=1e-12)
    assert ((g <= f) & (g >= f / 8 * (1 - 1e-12))).all()
    g, _ = rotary.rotary_frequencies(2, scaling="ntk", factor=8.0)   # one pair: nothing to spread over
    assert g.item() == 1 / 8


def test_yarn_keeps_fast_pairs_and_divides_slow_ones():
    f, _ = rotary.rotary_frequencies(128)
    g, s = rotary.rotary_frequencies(128, scaling="yarn", factor=4.0, original_length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert s == pytest.approx(0.1 * math.log(4.0) + 1.0)
    assert torch.equal(g[turns > 64], f[turns > 64])             # well above beta_fast = 32
    assert torch.allclose(g[turns < 0.5], f[turns < 0.5] / 4, rtol=1e-15, atol=0)
    between = (turns > 1.5) & (turns < 25)
    assert between.any() and ((g < f) & (g > f / 4))[between].all()


def test_axial_frequencies_and_grid_positions():
    f, axes = rotary.axial_frequencies(128)
    assert axes == (22, 21, 21) and f.numel() == 64
    assert f[0] == f[22] == f[43] == 1.0
    assert f[23].item() == pytest.approx(10000.0 ** (-2 / 42), rel=1e-15)
    p = rotary.grid_positions(2, 3, 4)
    want = [[t, h, w] for t in range(2) for h in range(3) for w in range(4)]
    assert p.t().tolist() == want


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"),
                                dict(rotary_dim=8, factor=2.0), dict(rotary_dim=8, scaling="linear", factor=0.5),
                                dict(rotary_dim=8, scaling="yarn", factor=2.0), dict(rotary_dim=8, theta=-1.0),
                                dict(rotary_dim=8, scaling="yarn", factor=2.0, original_length=64, theta=0.5)])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        rotary.rotary_frequencies(**kw)


def test_axial_and_grid_refusals():
    with pytest.raises(ValueError):
        rotary.axial_frequencies(4)
    with pytest.raises(ValueError):
        rotary.grid_positions(2, 0, 4)


# ---- refusals of the front ends ---------------------------------------------------
def _spec(B=2, N=5, d=8, device="cpu", **kw):
    kw.setdefault("inv_freq", torch.ones(4, dtype=torch.float64))
    return b.spa2_rotary_spec.from_buffer_copy(rotary._spec(rotary.Rotary(**kw), B, N, d, torch.device(device))[0])


def test_rotary_spec_marshalling():
    pos = torch.arange(40, dtype=torch.int32).view(2, 2, 10)[..., ::2]
    s = _spec(positions=pos, axes=(1, 3), layout="half", scale=1.5)
    assert (s.position_bytes, s.axes, list(s.pairs)[:2], s.rotary_dim, s.layout) == (4, 2, [1, 3], 8, b.ROTARY_HALF)
    assert list(s.position_stride) == [20, 10, 2] and s.scale == 1.5
    assert list(_spec(positions=torch.arange(5)).position_stride) == [0, 0, 1]
    assert list(_spec(positions=torch.zeros(2, 5, dtype=torch.int64)).position_stride) == [5, 0, 1]
    assert _spec().positions is None


@pytest.mark.parametrize("error,kw", [
    (ValueError, dict(layout="pairs")),
    (TypeError, dict(inv_freq=torch.ones(4))),
    (TypeError, dict(inv_freq=torch.ones(2, 2, dtype=torch.float64))),
    (ValueError, dict(inv_freq=torch.ones(0, dtype=torch.float64))),
    (ValueError, dict(inv_freq=torch.ones(5, dtype=torch.float64))),
    (ValueError, dict(inv_freq=torch.ones(4, dtype=torch.float64, requires_grad=True))),
    (ValueError, dict(axes=(1, 2), positions=torch.zeros(2, 5, dtype=torch.int64))),
    (ValueError, dict(axes=(5, -1), positions=torch.zeros(2, 5, dtype=torch.int64))),
    (ValueError, dict(axes=(1, 1, 1, 1, 0), positions=torch.zeros(5, 5, dtype=torch.int64))),
    (ValueError, dict(axes=())),
    (ValueError, dict(axes=(2, 2))),
    (ValueError, dict(scale=math.nan)),
    (TypeError, dict(positions=torch.zeros(5))),
    (ValueError, dict(positions=torch.zeros(4, dtype=torch.int64))),
    (ValueError, dict(positions=torch.zeros(3, 5, dtype=torch.int64))),
    (ValueError, dict(positions=torch.zeros(5, dtype=torch.int64), device="cuda:0")),
])
def test_rotary_refusals(error, kw):
    with pytest.raises(error):
        _spec(**kw)


def test_apply_rotary_refusals():
    f = torch.ones(4, dtype=torch.float64)
    q = torch.zeros(2, 3, 5, 8)
    for error, args in [(TypeError, (q.double(),)), (TypeError, (q, q.half())), (ValueError, (q[0],)),
                        (ValueError, (q, q[:1])), (ValueError, (q, q[:, :, :4])), (ValueError, (q, q[..., :6])),
                        (ValueError, (q, q))]:   # the last: not on a CUDA device
        with pytest.raises(error):
            rotary.apply_rotary(*args, inv_freq=f)


def test_pack8_refusals():
    x = torch.zeros(2, 8)
    for error, args in [(ValueError, ()), (TypeError, (x.int(),)), (TypeError, (x, x.half())), (ValueError, (x,)),
                        (ValueError, (torch.tensor(1.0),))]:
        with pytest.raises(error):
            checkpoint.pack8(*args)
    with pytest.raises(ValueError):
        checkpoint.unpack8()
    p = checkpoint.Packed.empty_like
    with pytest.raises(TypeError):
        checkpoint.unpack8(p(x), p(x.half()))


def test_packed_layout():
    p = checkpoint.Packed.empty_like(torch.zeros(3, 2, 33, dtype=torch.bfloat16))
    assert p.codes.shape == (3, 2, 33) and p.codes.dtype == torch.int8
    assert p.exponents.shape == (3, 2, 2) and p.nbytes == 208 + 12      # 198 codes, 16-byte aligned exponents
    assert p.exponents.data_ptr() == p.codes.data_ptr() + 208
    e = checkpoint.Packed.empty_like(torch.zeros(0, 4))
    assert e.codes.shape == (0, 4) and e.exponents.shape == (0, 1) and e.nbytes == 0


def test_several_checkpoints_in_one_buffer():
    x = torch.zeros(3, 33, dtype=torch.bfloat16)      # 99 codes, 112 with the padding, and 6 exponents
    kept = checkpoint.Packed.several_like(x, 3)
    assert kept[0].base.numel() == 3 * 128 and [p.offset for p in kept] == [0, 128, 256]
    for p in kept:
        assert p.nbytes == 118 and p.data.numel() == 118 and p.codes.shape == (3, 33) and p.exponents.shape == (3, 2)
        assert p.codes.data_ptr() == p.base.data_ptr() + p.offset and p.fields()[1:3] == (
            p.codes.data_ptr(), p.exponents.data_ptr())
    again = checkpoint.Packed.several_in(kept[0].base, x.shape, x.dtype, 3)
    assert [p.fields() for p in again] == [p.fields() for p in kept]


def test_status_fetch_argument_errors(L):
    assert L.spa2_status_fetch(None, FAKE, None) == b.ERR_WORKSPACE
    assert L.spa2_status_fetch(FAKE, None, None) == L.spa2_status_fetch(FAKE, FAKE + 2, None) == b.ERR_INVALID_ARG


def test_packed_rotary_spec_points_at_its_tensors():
    f, pos = torch.ones(4, dtype=torch.float64), torch.arange(5)
    spec, _ = rotary._spec(rotary.Rotary(f, pos), 2, 5, 8, torch.device("cpu"))
    assert b.rotary_spec_points(spec, f, pos)
    assert not b.rotary_spec_points(spec, f.clone(), pos) and not b.rotary_spec_points(spec, f, pos.clone())
    assert not b.rotary_spec_points(spec, f, None)
    every_other = torch.ones(8, dtype=torch.float64)[::2]      # copied for the call: not to be kept
    spec, copy = rotary._spec(rotary.Rotary(every_other, pos), 2, 5, 8, torch.device("cpu"))
    assert copy.is_contiguous() and not b.rotary_spec_points(spec, every_other, pos)


def test_sparse_attention_checkpoint_refusals():
    q = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        autograd.sparse_attention(q, q, q, checkpoint="fp8")
    for error, args in [(TypeError, (q, q, q.float())), (ValueError, (q, q[:, :, :64], q)), (ValueError, (q, q, q[:, :1])),
                        (ValueError, (q[0], q[0], q[0])), (ValueError, (q, q, q))]:
        with pytest.raises(error):
            autograd.sparse_attention(*args, checkpoint="int8")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = (i(1, 2, 1), i(1, 2, 1, 2), i(1, 2, 2), i(1, 2, 2, 1))
    fake = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16, device="meta")
    for n, t in enumerate((i(1, 2, 2), i(1, 2, 1, 3), None, i(1, 2, 2, 1).long())):
        mask = b.Mask(*good[:n], t, *good[n + 1:])
        with pytest.raises(ValueError):
            autograd._check_attention(q, q, q, mask, b.BQ, b.BKV)
    with pytest.raises(ValueError):
        autograd._check_attention(fake, fake, fake, b.Mask(*good), b.BQ, b.BKV)


# ---- refusals of the C entry points -----------------------------------------------
FAKE = 1 << 20   # never dereferenced: validation fails first


def _rotary_call(n=1, B=1, N=4, d=8, dtype=b.DTYPE_BF16, x=FAKE, y=FAKE, heads=2, null_spec=False, **kw):
    t = (b.spa2_rotary_tensor * 3)()
    for e in t:
        e.x, e.y, e.heads = x, y, heads
    s = b.spa2_rotary_spec()
    s.position_bytes, s.axes, s.inv_freq, s.rotary_dim, s.layout, s.scale = 8, 1, FAKE, 8, 0, 1.0
    s.pairs[0] = 4
    for name, v in kw.items():
        if name == "pairs":
            s.pairs[:] = v
        else:
            setattr(s, name, v)
    return b.lib().spa2_rotary(t, n, B, N, d, dtype, None if null_spec else ctypes.byref(s), 0, None)


@pytest.mark.parametrize("want,kw", [
    (b.ERR_INVALID_ARG, dict(n=0)), (b.ERR_INVALID_ARG, dict(B=0)), (b.ERR_INVALID_ARG, dict(N=-1)),
    (b.ERR_INVALID_ARG, dict(x=None)), (b.ERR_INVALID_ARG, dict(y=FAKE + 1)), (b.ERR_INVALID_ARG, dict(heads=0)),
    (b.ERR_INVALID_ARG, dict(inv_freq=None)), (b.ERR_INVALID_ARG, dict(inv_freq=FAKE + 4)),
    (b.ERR_INVALID_ARG, dict(positions=FAKE + 4)), (b.ERR_INVALID_ARG, dict(null_spec=True)),
    (b.ERR_INVALID_ARG, dict(pairs=[3, 0, 0, 0])), (b.ERR_INVALID_ARG, dict(pairs=[-1, 5, 0, 0], axes=2, positions=FAKE)),
    (b.ERR_UNSUPPORTED, dict(n=3)), (b.ERR_UNSUPPORTED, dict(d=1026)), (b.ERR_UNSUPPORTED, dict(rotary_dim=7)),
    (b.ERR_UNSUPPORTED, dict(rotary_dim=10)), (b.ERR_UNSUPPORTED, dict(axes=5)), (b.ERR_UNSUPPORTED, dict(dtype=9)),
    (b.ERR_UNSUPPORTED, dict(layout=2)), (b.ERR_UNSUPPORTED, dict(positions=FAKE, position_bytes=2)),
    (b.ERR_UNSUPPORTED, dict(axes=2, pairs=[2, 2, 0, 0])), (b.ERR_UNSUPPORTED, dict(B=65536, N=65536)),
    (b.ERR_UNSUPPORTED, dict(heads=65536)), (b.ERR_INVALID_ARG, dict(dtype=b.DTYPE_F32, x=FAKE + 2)),
])
def test_rotary_argument_errors(want, kw):
    assert _rotary_call(**kw) == want


@pytest.mark.parametrize("call", ["spa2_pack8", "spa2_unpack8"])
def test_pack8_argument_errors(L, call):
    f = getattr(L, call)

    def go(n=1, dtype=b.DTYPE_BF16, **kw):
        t = (b.spa2_pack8_tensor * 9)(*(b.spa2_pack8_tensor(FAKE, FAKE, FAKE, 4, 64) for _ in range(9)))
        for name, v in kw.items():
            setattr(t[0], name, v)
        return f(t, n, dtype, None)

    assert f(None, 1, 0, None) == b.ERR_INVALID_ARG
    for kw in (dict(n=0), dict(x=None), dict(codes=None), dict(exps=None), dict(x=FAKE + 1), dict(rows=-1), dict(d=0)):
        assert go(**kw) == b.ERR_INVALID_ARG, kw
    for kw in (dict(n=9), dict(dtype=5), dict(rows=1 << 40)):
        assert go(**kw) == b.ERR_UNSUPPORTED, kw
    assert go(rows=0, x=None, codes=None, exps=None) == b.OK     # nothing to do, nothing launched


def test_checkpointed_attention_argument_errors():
    m = b.spa2_mask(FAKE, FAKE, FAKE, FAKE, None, None)
    ok = b.spa2_pack8_tensor(None, FAKE, FAKE, 0, 0)
    bad = [b.spa2_pack8_tensor(None, None, FAKE, 0, 0), b.spa2_pack8_tensor(None, FAKE, None, 0, 0),
           b.spa2_pack8_tensor(None, FAKE + 8, FAKE, 0, 0), b.spa2_pack8_tensor(None, FAKE, FAKE + 2, 0, 0)]
    fwd = lambda q=FAKE, N=128, d=128, bq=128, scale=0.0, o=FAKE, lse=None, p=(ok, ok, ok), n=1 << 30, mask=m: (  # noqa: E731
        b.spa2_sparse_attn_fwd_ckpt(q, FAKE, FAKE, 1, 1, N, d, bq, 64, mask, scale, o, lse, *p, FAKE, n, None))
    bwd = lambda dout=FAKE, N=128, d=128, bq=128, scale=0.0, dq=FAKE, dt=0, p=(ok, ok, ok), n=1 << 30, mask=m: (  # noqa: E731
        b.spa2_sparse_attn_bwd_ckpt(*p, dout, 1, 1, N, d, bq, 64, mask, scale, dq, FAKE, FAKE, dt, FAKE, n, None))
    for x in bad:
        for i in range(3):
            p = [ok, ok, ok]
            p[i] = x
            assert fwd(p=p) == b.ERR_INVALID_ARG and bwd(p=p) == b.ERR_INVALID_ARG
    half = b.spa2_mask(FAKE, FAKE, None, None, None, None)
    assert bwd(mask=half) == b.ERR_INVALID_ARG                        # the backward needs the columns
    assert fwd(q=None) == fwd(q=FAKE + 2) == fwd(o=None) == fwd(lse=FAKE + 2) == b.ERR_INVALID_ARG
    assert bwd(dout=None) == bwd(dout=FAKE + 2) == bwd(dq=FAKE + 8) == b.ERR_INVALID_ARG
    assert fwd(N=0) == bwd(N=0) == b.ERR_INVALID_ARG
    for call in (fwd, bwd):
        assert call(d=96) == call(bq=96) == call(N=131073) == call(scale=-1.0) == call(scale=math.inf) == b.ERR_UNSUPPORTED
        assert call(n=300) == b.ERR_WORKSPACE
    assert bwd(dt=b.DTYPE_F16) == b.ERR_UNSUPPORTED


def test_checkpoint_workspace_holds_lse_and_kept_values():
    for N, d, bq in ((32760, 128, 128), (1000, 64, 64), (1, 64, 256)):
        n = b.spa2_workspace_bytes(b.OP_BWD_CKPT, 1, 2, N, d, bq)
        assert n >= b.spa2_workspace_bytes(b.OP_BWD, 1, 2, N, d, bq) + 2 * N * (4 + 2 * 2 * d)
    assert b.spa2_workspace_bytes(b.OP_BWD_CKPT, 1, 2, 100, 96) == 0
