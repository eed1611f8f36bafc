"""8-bit checkpoints on the GPU: pack8 / unpack8 against the definition (exact), and
attention that trains on checkpoints against the float64 oracle at the kept values."""

import math

import numpy as np
import pytest
import torch

import oracle
from tests._parity import assert_close, assert_close_bf16_out, bf16_half_ulp, csr_to_dense, f64
from trainable_block_sparse_pooled_b200 import binding as b
from trainable_block_sparse_pooled_b200 import synth
from trainable_block_sparse_pooled_b200.autograd import block_mask, check_errors, sparse_attention
from trainable_block_sparse_pooled_b200.checkpoint import pack8, unpack8
from trainable_block_sparse_pooled_b200.rotary import Rotary, apply_rotary, axial_frequencies, grid_positions

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def kept(x):
    """(codes, exponents, values) of x [..., d] by the definition, in NumPy float64."""
    x = x.detach().double().cpu().numpy()
    d = x.shape[-1]
    y = np.zeros(x.shape[:-1] + (-(-d // 32) * 32,))
    y[..., :d] = x
    y = y.reshape(x.shape[:-1] + (y.shape[-1] // 32, 32))
    most = np.abs(y).max(-1)
    with np.errstate(invalid="ignore"):
        finite = np.isfinite(most)
        E = np.where(finite, np.clip(np.frexp(np.where(finite, most, 0.0))[1] - 1 + 127, 0, 254), 255)
        E = np.where(most == 0, 0, E)
        scaled = np.ldexp(np.where(np.isfinite(y), y, 0.0), (133 - E)[..., None])
    codes = np.clip(np.rint(scaled), -127, 127)
    values = np.where((E == 255)[..., None], np.nan, np.ldexp(codes, (E - 133)[..., None]))
    flat = lambda t: t.reshape(x.shape[:-1] + (t.shape[-2] * 32,))[..., :d]  # noqa: E731
    return flat(codes), E, flat(values)


def check(x):
    (p,) = pack8(x)
    (y,) = unpack8(p)
    codes, E, values = kept(x)
    assert y.dtype == x.dtype and y.shape == x.shape and y.is_contiguous()
    assert np.array_equal(p.exponents.cpu().numpy(), E)
    assert np.array_equal(y.double().cpu().numpy(), values, equal_nan=True)
    fine = ~np.isnan(values)
    assert np.array_equal(p.codes.cpu().numpy()[fine], codes[fine])
    return p


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1,), (31,), (3, 32), (5, 33), (2, 3, 40), (257, 64), (7, 100), (4, 128), (3, 1000),
                                   (1, 5120), (2049, 8), (33, 1536)])
def test_values_are_those_of_the_definition(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randn(shape, generator=g, device="cuda")
    x = x * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    x[..., ::7] *= 30
    check(x.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_every_16_bit_value(dtype):
    """All finite bit patterns, each the largest of its group and each beside larger ones."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    bits = bits[torch.isfinite(bits)].cuda()
    x = bits[:, None] * torch.ones(32, device="cuda", dtype=dtype)
    x[:, 1:] = bits[torch.randint(0, bits.numel(), (bits.numel(), 31), generator=torch.Generator().manual_seed(1))]
    check(torch.where(x.float().abs() <= bits[:, None].float().abs(), x, torch.zeros_like(x)))
    check(x)


def test_ties_limits_and_subnormals():
    x = torch.zeros(12, 32, dtype=F32)
    x[0, :4] = torch.tensor([64.0, 0.5, 1.5, -2.5])                 # ties go to the even code
    x[1, :4] = torch.tensor([127.5, 127.4, -127.5, 126.5])          # 127.5 rounds to 128: clamped
    x[2, :2] = torch.tensor([127.99999, -127.99999])
    x[3, :3] = torch.tensor([3.4028234663852886e38, -1e38, 1e36])   # the largest exponent, 254
    x[4, :3] = torch.tensor([1.401298464324817e-45, 0.0, -1e-40])   # subnormals
    x[5, :2] = torch.tensor([1.1754943508222875e-38, 1e-39])        # the smallest normal, E = 1
    x[6, :2] = torch.tensor([2.0 ** -120, -2.0 ** -127])
    x[7] = -0.0
    x[8, 5] = math.nan
    x[9, 31] = math.inf
    x[10, 0] = -math.inf
    x[11] = 1.0
    p = check(x.cuda())
    assert p.exponents[:, 0].tolist()[7:] == [0, 255, 255, 255, 127]
    assert p.exponents[3, 0] == 254 and p.exponents[5, 0] == 1
    check(x.to(BF16).cuda())


def test_infinities_and_nan_stay_in_their_group():
    x = torch.randn(40, 100, device="cuda").to(BF16)
    (want,) = unpack8(*pack8(x))
    bad = x.clone()
    bad[3, 40], bad[7, 99], bad[9, 0] = math.nan, math.inf, -math.inf
    (got,) = unpack8(*pack8(bad))
    lost = torch.zeros(40, 100, dtype=torch.bool, device="cuda")
    lost[3, 32:64], lost[7, 96:], lost[9, :32] = True, True, True
    assert torch.isnan(got[lost]).all() and torch.equal(got[~lost], want[~lost])


def test_strides_offsets_and_many_tensors():
    xs = [torch.randn(40, 64, device="cuda").to(BF16).t(), torch.randn(3, 5, 72, device="cuda").to(BF16)[:, ::2, 4:68],
          torch.randn(129, device="cuda").to(BF16)[1:], torch.randn(5, 36, device="cuda").to(BF16).flatten()[4:148].view(4, 36),
          torch.randn(1, 64, device="cuda").to(BF16).expand(6, -1), torch.zeros(0, 64, device="cuda", dtype=BF16),
          torch.zeros(4, 0, 64, device="cuda", dtype=BF16)]
    xs += [torch.randn(n, 8 * n, device="cuda").to(BF16) for n in range(1, 13)]
    packed = pack8(*xs)
    for x, p, y in zip(xs, packed, unpack8(*packed)):
        assert p.nbytes <= 1.04 * x.numel() + 16 + x.numel() // max(1, min(32, x.shape[-1]))
        assert torch.equal(y, torch.from_numpy(kept(x)[2]).to(BF16).cuda())


def test_a_checkpoint_of_kept_values_is_itself():
    x = torch.randn(64, 256, device="cuda").to(BF16)
    (y,) = unpack8(*pack8(x))
    (z,) = unpack8(*pack8(y))
    assert torch.equal(y, z)


def test_more_than_2_31_elements():
    rows, d = 2 ** 25 + 3, 64
    x = torch.zeros(rows, d, dtype=BF16, device="cuda")
    x[-5:] = torch.randn(5, d, device="cuda").to(BF16)
    x[:5] = torch.randn(5, d, device="cuda").to(BF16)
    (p,) = pack8(x)
    (y,) = unpack8(p)
    for part in (slice(0, 5), slice(rows - 5, rows)):
        assert np.array_equal(y[part].double().cpu().numpy(), kept(x[part])[2])
    assert not y[5:-5].any()


def test_rows_behind_the_last_are_left():
    """The C entry points write rows * d codes, rows * ceil(d / 32) exponents and rows * d values, nothing more."""
    for d in (64, 40, 33):
        for rows in (1, 5, 70):
            x = torch.randn(rows, d, device="cuda").to(BF16)
            codes = torch.full((rows * d + 64,), 99, dtype=torch.int8, device="cuda")
            exps = torch.full((rows * -(-d // 32) + 64,), 77, dtype=torch.uint8, device="cuda")
            y = torch.full((rows * d + 64,), 55.0, dtype=BF16, device="cuda")
            s = torch.cuda.current_stream().cuda_stream
            for call, t in ((b.spa2_pack8, x), (b.spa2_unpack8, y)):
                item = b.spa2_pack8_tensor(t.data_ptr(), codes.data_ptr(), exps.data_ptr(), rows, d)
                assert call((b.spa2_pack8_tensor * 1)(item), b.DTYPE_BF16, s) == b.OK
            assert (codes[rows * d:] == 99).all() and (exps[rows * -(-d // 32):] == 77).all()
            assert (y[rows * d:] == 55.0).all() and torch.equal(y[:rows * d].view(rows, d), unpack8(*pack8(x))[0])


def test_pack_on_a_side_stream_and_captured():
    x = torch.randn(300, 128, device="cuda").to(BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        (y,) = unpack8(*pack8(x))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, unpack8(*pack8(x))[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (y,) = unpack8(*pack8(x))
    x.copy_(torch.randn_like(x))
    graph.replay()
    assert torch.equal(y, unpack8(*pack8(x))[0])


# ---- attention on checkpoints --------------------------------------------------------
def attention(q, k, v, dout, mask, bq=b.BQ, bkv=b.BKV, **kw):
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = sparse_attention(*leaves, mask=mask, bq=bq, bkv=bkv, checkpoint="int8", **kw)
    return (o.detach(), *torch.autograd.grad(o, leaves, dout))


def against_oracle(q, k, v, dout, mask, bq=b.BQ, bkv=b.BKV, scale=0.0, **kw):
    """o of the inputs, gradients at the kept values."""
    got = attention(q, k, v, dout, mask, bq, bkv, scale=scale, **kw)
    check_errors()
    assert torch.equal(got[0], sparse_attention(q, k, v, mask=mask, bq=bq, bkv=bkv, scale=scale))
    dense = csr_to_dense(mask.row_cnt.cpu().numpy(), mask.row_idx.cpu().numpy(), mask.row_idx.shape[-1])
    q8, k8, v8 = (kept(x)[2] for x in (q, k, v))
    more = (scale,) if scale else ()
    want = oracle.masked_attn_bwd(q8, k8, v8, dense, f64(dout), bq, bkv, *more)
    for name, g, e in zip(("dQ", "dK", "dV"), got[1:], want):
        assert g.dtype == BF16
        assert_close_bf16_out(f64(g), e, name)
    return got


@pytest.mark.parametrize("B,H,N,d,bq,bkv", [
    (1, 2, 512, 64, 128, 64), (1, 2, 1000, 128, 128, 64), (2, 1, 1000, 64, 64, 128), (1, 1, 130, 128, 256, 64),
    (1, 3, 63, 64, 64, 64), (2, 2, 65, 128, 256, 128), (1, 1, 127, 64, 128, 128), (1, 1, 2049, 128, 128, 64)])
def test_gradients_match_the_oracle_at_the_kept_values(B, H, N, d, bq, bkv):
    q, k, v = synth.gaussian_with_sinks(B=B, H=H, N=N, d=d, seed=N + d, device="cuda")
    dout = synth.normal_like(q.shape, seed=N, device="cuda")
    against_oracle(q, k, v, dout, block_mask(q, k, 0.2, 0.6, bq, bkv), bq, bkv)


@pytest.mark.parametrize("N", [1, 2, 64])
def test_short_sequences(N):
    q, k, v = (synth.normal_like((2, 3, N, 64), seed=i, device="cuda") for i in range(3))
    dout = synth.normal_like(q.shape, seed=9, device="cuda")
    o, dq, dk, dv = against_oracle(q, k, v, dout, block_mask(q, k, 1.0, 1.0))
    if N == 1:   # one key: o = v, and dv = dout
        assert torch.equal(o, v) and torch.equal(dv, dout)


def test_gradients_against_differences():
    """<dq, u> + <dk, u'> + <dv, u''> against central differences of <o, dout> of the
    oracle at the kept values: the differences are off by O(h^2) (h = 1e-4: 1e-7
    relative), the gradients by at most 2e-2 and half a bf16 step each; over the n
    elements of a random direction of +-1 the errors add up to at most that sum."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=256, d=64, seed=5, device="cuda")
    dout = synth.normal_like(q.shape, seed=6, device="cuda")
    mask = block_mask(q, k, 0.4, 0.6)
    grads = attention(q, k, v, dout, mask)[1:]
    dense = csr_to_dense(mask.row_cnt.cpu().numpy(), mask.row_idx.cpu().numpy(), mask.row_idx.shape[-1])
    at = [kept(x)[2] for x in (q, k, v)]
    rng = np.random.default_rng(7)
    loss = lambda xs: float((oracle.masked_attn_fwd(*xs, dense, 128, 64)[0] * f64(dout)).sum())  # noqa: E731
    for i, g in enumerate(grads):
        u = rng.choice((-1.0, 1.0), size=at[0].shape)
        h = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * u, at[i] - h * u
        want = (loss(up) - loss(down)) / (2 * h)
        # per element the kernel's error is far below the 2e-2 bound: 1e-2 relative L1 as well
        bound = 1e-2 * np.abs(f64(g)).sum() + bf16_half_ulp(f64(g)).sum() + 1e-5 * abs(want)
        assert abs(float((f64(g) * u).sum()) - want) <= bound


def test_own_mask_scale_and_return_mask():
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=700, d=64, seed=8, device="cuda")
    dout = synth.normal_like(q.shape, seed=9, device="cuda")
    m = block_mask(q, k, 0.2, 0.6)
    against_oracle(q, k, v, dout, m, scale=0.2)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o, cnt = sparse_attention(*leaves, k_frac=0.2, p_frac=0.6, checkpoint="int8", return_mask=True)
    assert torch.equal(cnt, m.row_cnt) and not cnt.requires_grad
    got = torch.autograd.grad(o, leaves, dout)
    assert all(torch.equal(a, c) for a, c in zip(got, attention(q, k, v, dout, m)[1:]))


def test_only_8_bits_are_kept_and_a_second_backward_is_refused():
    q, k, v = (x.requires_grad_() for x in synth.gaussian_with_sinks(B=1, H=2, N=2000, d=128, seed=1, device="cuda"))
    m = block_mask(q.detach(), k.detach(), 0.2, 0.6)
    sparse_attention(q, k, v, mask=m, checkpoint="int8").sum().backward()   # workspaces exist from here on
    torch.cuda.synchronize()
    requested = lambda: torch.cuda.memory_stats()["requested_bytes.all.current"]  # noqa: E731  (not the allocator's blocks)
    before = requested()
    o = sparse_attention(q, k, v, mask=m, checkpoint="int8")
    torch.cuda.synchronize()
    kept_bytes = requested() - before - o.numel() * 2
    assert kept_bytes <= 3 * 33 / 32 * q.numel() + 16384
    loss = o.float().sum()
    loss.backward()
    with pytest.raises(RuntimeError):
        loss.backward()


def test_a_second_derivative_is_refused():
    """create_graph gives the same gradients; differentiating them again raises."""
    q, k, v = (x.requires_grad_() for x in synth.gaussian_with_sinks(B=1, H=1, N=300, d=64, seed=27, device="cuda"))
    m = block_mask(q.detach(), k.detach(), 0.3, 0.5)
    dout = synth.normal_like(q.shape, seed=28, device="cuda").requires_grad_()
    o = sparse_attention(q, k, v, mask=m, checkpoint="int8")
    grads = torch.autograd.grad(o, (q, k, v), dout, create_graph=True)
    assert all(torch.equal(a, w) for a, w in zip(grads, attention(q, k, v, dout.detach(), m)[1:]))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(grads[0].float().sum(), q)


def test_no_gradient_keeps_nothing():
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=300, d=64, seed=2, device="cuda")
    m = block_mask(q, k, 0.3, 0.5)
    o = sparse_attention(q, k, v, mask=m, checkpoint="int8")
    assert not o.requires_grad and torch.equal(o, sparse_attention(q, k, v, mask=m))
    with torch.no_grad():
        assert sparse_attention(q.requires_grad_(), k, v, mask=m, checkpoint="int8").grad_fn is None


def test_strided_inputs_and_broadcast_gradient():
    """Views of projections, and a gradient that is an expanded scalar."""
    x = synth.normal_like((2, 200, 3, 2, 64), seed=3, device="cuda")
    q, k, v = (x[:, :, i].transpose(1, 2).detach().requires_grad_() for i in range(3))
    m = block_mask(q.detach(), k.detach(), 0.5, 0.5)
    o = sparse_attention(q, k, v, mask=m, checkpoint="int8")
    got = torch.autograd.grad(o.sum(), (q, k, v))
    want = attention(q.contiguous(), k.contiguous(), v.contiguous(), torch.ones(2, 2, 200, 64, device="cuda", dtype=BF16), m)
    assert all(torch.equal(a, c) for a, c in zip(got, want[1:]))


def test_nan_in_keys_that_no_query_keeps():
    """A key block that the mask leaves out may hold anything: o, dq and the kept
    blocks' gradients do not see it, its own gradients are zero."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=512, d=64, seed=4, device="cuda")
    dout = synth.normal_like(q.shape, seed=5, device="cuda")
    keep = torch.zeros(4, 8, dtype=torch.bool)
    keep[:, [0, 2, 3, 6]] = True
    ids = torch.tensor([0, 2, 3, 6, 7, 7, 7, 7], dtype=torch.int32)
    cols = torch.tensor([4, 0, 4, 4, 0, 0, 4, 0], dtype=torch.int32)
    m = b.Mask(torch.full((1, 1, 4), 4, dtype=torch.int32).cuda(), ids.repeat(1, 1, 4, 1).cuda(), cols.view(1, 1, 8).cuda(),
               torch.arange(4, dtype=torch.int32).repeat(1, 1, 8, 1).cuda())
    want = attention(q, k, v, dout, m)
    check_errors()
    for block, value in ((1, math.nan), (4, -math.inf), (5, 1e-30), (7, 3e38)):
        k[0, 0, block * 64:block * 64 + 64] = value
    got = attention(q, k, v, dout, m)
    check_errors()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    off = torch.cat([torch.arange(j * 64, j * 64 + 64) for j in (1, 4, 5, 7)])
    assert not got[2][0, 0, off].any() and not got[3][0, 0, off].any()


def test_values_beyond_fp16_are_reported():
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=256, d=64, seed=6, device="cuda")
    dout = synth.normal_like(q.shape, seed=7, device="cuda")
    m = block_mask(q, k, 1.0, 1.0)
    check_errors()
    for at in range(3):   # not dout: it is scaled
        args = [q.clone(), k.clone(), v.clone(), dout.clone()]
        args[at][0, 0, 3, 3] = 1e6
        with pytest.raises(b.Spa2Error) as e:   # by the backward pass if the copy has landed, else by check_errors
            attention(*args, m)
            check_errors()
        assert e.value.code == b.ERR_RANGE
    attention(q, k, v, dout, m)
    check_errors()


def test_gradients_scale_with_dout():
    """Gradients are linear in dout: powers of two per head come through bit for bit, from gradients
    of 1e-9 to ones of 1e6 (bf16 has the range; a half would not)."""
    q, k, v = synth.gaussian_with_sinks(B=2, H=3, N=700, d=64, seed=17, device="cuda")
    dout = synth.normal_like(q.shape, seed=18, device="cuda")
    m = block_mask(q, k, 0.3, 0.6)
    want = attention(q, k, v, dout, m)[1:]
    powers = torch.tensor([[0, -30, 20], [-12, 7, -60]], device="cuda")[..., None, None]
    got = attention(q, k, v, torch.ldexp(dout.float(), powers).to(BF16), m)[1:]
    check_errors()
    for a, w in zip(got, want):
        assert torch.equal(a, torch.ldexp(w.float(), powers).to(BF16))
    zero = attention(q, k, v, torch.zeros_like(dout), m)[1:]
    assert not any(x.any() for x in zero)


def test_large_values():
    """v times 2^8 or 2^11 gives dq and dk times as much and the same dv, where dS would leave a half's range
    if dO kept its own. dO is scaled down by up to 2^10 then: its small elements lose at most
    2^-25 of a largest of 2^-7 or more, and dS as much, 4e-6 of the largest; the results may round to the
    other neighbour, one bf16 step (twice half a step), and near zero differ by 1e-4 of the largest."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=512, d=128, seed=25, device="cuda")
    dout = synth.normal_like(q.shape, seed=26, device="cuda")
    m = block_mask(q, k, 0.4, 0.6)
    want = attention(q, k, v, dout, m)[1:]
    for power in (8, 11):
        got = attention(q, k, torch.ldexp(v.float(), torch.tensor(power, device="cuda")).to(BF16), dout, m)[1:]
        check_errors()
        for a, w, times in zip(got, want, (2.0 ** -power, 2.0 ** -power, 1.0)):
            a, w = f64(a) * times, f64(w)
            assert np.isfinite(a).all()
            assert (np.abs(a - w) <= 2 * bf16_half_ulp(w) + 1e-4 * np.abs(w).max()).all()


def test_small_rows_beside_large_ones():
    """Rows of dout at 2^-12 of the others: what they alone contribute, the values' gradients of a key
    block that only they keep. With the head's largest |dout| in [4, 8) (here it is: no scaling)
    their fp16 elements are exact from 2^-17 up and off by at most 2^-25 below; over the 128 rows,
    with P <= 1, that adds up to 2^-18. Both results are rounded to bf16, 2^-9 each of the value
    (half a step is 2^-8 of a power of two, 2^-9 to 2^-8 relative)."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=512, d=64, seed=19, device="cuda")
    dout = synth.normal_like(q.shape, seed=20, device="cuda")
    small = dout.clone()
    small[0, 0, 256:384] *= 2.0 ** -12
    keep = torch.ones(1, 1, 4, 8, dtype=torch.bool)
    keep[..., 5] = False
    keep[0, 0, 2] = False
    keep[0, 0, 2, 5] = True            # the third query block keeps the sixth key block, which nobody else does
    m = lists(keep)
    assert 4 <= small.abs().max() < 8
    dv, dv_small = (attention(q, k, v, x, m)[3][0, 0, 320:384].double() for x in (dout, small))
    assert ((dv_small - dv * 2.0 ** -12).abs() <= 2.0 ** -18 + 2 * 2.0 ** -8 * dv.abs() * 2.0 ** -12).all()
    assert dv.abs().median() > 0.1   # 2.4e-5 of the small rows: six times what the sum allows


def test_infinite_gradients_are_reported():
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=256, d=64, seed=21, device="cuda")
    m = block_mask(q, k, 1.0, 1.0)
    for bad in (math.inf, math.nan):
        dout = synth.normal_like(q.shape, seed=22, device="cuda")
        dout[0, 1, 100, 3] = bad
        check_errors()
        with pytest.raises(b.Spa2Error) as e:
            attention(q, k, v, dout, m)
            check_errors()
        assert e.value.code == b.ERR_RANGE


def test_bad_masks_are_reported():
    """An empty row and an id behind the last block: reported, and nothing beyond the buffers is touched."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=384, d=64, seed=6, device="cuda")
    dout = synth.normal_like(q.shape, seed=7, device="cuda")
    good = block_mask(q, k, 1.0, 1.0)
    for name, at, value in (("row_cnt", (0, 0, 1), 0), ("row_idx", (0, 0, 1, 2), 6), ("col_cnt", (0, 0, 2), 4),
                            ("col_idx", (0, 0, 2, 1), 3)):
        m = b.Mask(*(t.clone() for t in (good.row_cnt, good.row_idx, good.col_cnt, good.col_idx)))
        getattr(m, name)[at] = value
        check_errors()
        with pytest.raises(b.Spa2Error) as e:
            attention(q, k, v, dout, m)
            check_errors()
        assert e.value.code == b.ERR_DEVICE_BOUNDS
        try:
            check_errors()
        except b.Spa2Error:
            pass
    attention(q, k, v, dout, good)
    check_errors()


def lists(keep):
    """The mask of a dense bool [B, H, T_m, T_n]."""
    def csr(x):
        n = x.shape[-1]
        ids = torch.where(x, torch.arange(n), n).sort(dim=-1).values.clamp(max=n - 1)
        return x.sum(-1).int().contiguous().cuda(), ids.int().contiguous().cuda()

    return b.Mask(*csr(keep), *csr(keep.transpose(-1, -2)))


@pytest.mark.parametrize("N,d,bq,bkv", [(1100, 128, 128, 64), (1100, 64, 128, 64), (1100, 64, 64, 64), (1030, 128, 256, 128)])
def test_every_count_of_kept_blocks(N, d, bq, bkv):
    """Row i keeps i + 1 blocks, then all of them: one tile, two, .. and the columns that nobody keeps."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=N, d=d, seed=N + bq, device="cuda")
    dout = synth.normal_like(q.shape, seed=N, device="cuda")
    Tm, Tn = b.block_counts(N, bq, bkv)
    keep = torch.zeros(1, 2, Tm, Tn, dtype=torch.bool)
    for i in range(Tm):
        keep[0, 0, i, :min(i + 1, Tn)] = True
        keep[0, 1, i, Tn - 1 - i % Tn] = True          # one block each; from the ragged last one on
        keep[0, 1, i, :i // 2] = True
    against_oracle(q, k, v, dout, lists(keep), bq, bkv)


@pytest.mark.parametrize("N,d,bq,bkv", [(4500, 64, 128, 64), (6000, 128, 128, 64), (4500, 128, 64, 64)])
def test_columns_that_every_query_block_keeps(N, d, bq, bkv):
    """Few heads and long columns: gathered from parts. The first block is kept by all query blocks, others by
    half, a quarter, an eighth of them and by one; the ragged last one by 33."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=1, N=N, d=d, seed=N + d, device="cuda")
    dout = synth.normal_like(q.shape, seed=N, device="cuda")
    Tm, Tn = b.block_counts(N, bq, bkv)
    keep = torch.zeros(1, 1, Tm, Tn, dtype=torch.bool)
    for column, step in ((0, 1), (1, 2), (2, 4), (3, 8)):
        keep[..., ::step, column] = True
    keep[0, 0, torch.arange(Tm), torch.arange(Tm) * bq // bkv] = True
    keep[..., :33, Tn - 1] = True
    m = lists(keep)
    got = against_oracle(q, k, v, dout, m, bq, bkv)
    assert all(torch.equal(a, c) for a, c in zip(got, attention(q, k, v, dout, m, bq, bkv)))
    s = b.Spa2(1, 1, N, d, bq=bq, bkv=bkv)
    grads = s.bwd_ckpt(pack8(q, k, v), dout, m)      # fp32
    s.check()
    assert all(torch.equal(a, c.to(BF16)) for a, c in zip(got[1:], grads))


def test_the_same_bits_when_all_columns_are_alike():
    """Every column is as long as every other: which of them are taken in parts must not depend on chance."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=3, N=4352, d=64, seed=23, device="cuda")
    dout = synth.normal_like(q.shape, seed=24, device="cuda")
    m = lists(torch.ones(1, 3, 34, 68, dtype=torch.bool))
    want = attention(q, k, v, dout, m)
    for _ in range(6):
        assert all(torch.equal(a, c) for a, c in zip(attention(q, k, v, dout, m), want))
    check_errors()


def test_more_than_2_31_elements_in_the_attention():
    """The last heads of a problem of more than 2^31 elements, against the same heads alone, bit for bit."""
    H, N, d = 130, 131072, 128
    Tm, Tn = b.block_counts(N)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, dout = (torch.zeros(1, H, N, d, dtype=BF16, device="cuda") for _ in range(4))
    for x in (q, k, v, dout):
        x[0, -2:] = torch.randn(2, N, d, generator=g, device="cuda").to(BF16)
    i, j = torch.arange(Tm, device="cuda", dtype=torch.int32), torch.arange(Tn, device="cuda", dtype=torch.int32)

    def mask(H):   # query block i keeps the two key blocks of its own rows
        m = b.Mask(torch.full((1, H, Tm), 2, dtype=torch.int32, device="cuda"),
                   torch.zeros(1, H, Tm, Tn, dtype=torch.int32, device="cuda"),
                   torch.ones(1, H, Tn, dtype=torch.int32, device="cuda"),
                   torch.zeros(1, H, Tn, Tm, dtype=torch.int32, device="cuda"))
        m.row_idx[..., 0], m.row_idx[..., 1], m.col_idx[..., 0] = 2 * i, 2 * i + 1, j // 2
        return m

    got = attention(q, k, v, dout, mask(H))
    want = attention(*(x[:, -2:].contiguous() for x in (q, k, v, dout)), mask(2))
    check_errors()
    assert all(torch.equal(a[:, -2:], w) for a, w in zip(got, want))
    assert all(w.float().abs().sum() > 0 for w in want) and not any(a[:, :-2].any() for a in got[1:])


def test_checkpoints_moved_to_the_host_and_back():
    """Saved tensors that come back at other addresses."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=500, d=64, seed=15, device="cuda")
    dout = synth.normal_like(q.shape, seed=16, device="cuda")
    inv_freq, axes = axial_frequencies(64, device="cuda")
    r = Rotary(inv_freq, grid_positions(5, 10, 10, device="cuda"), axes=axes)
    m = block_mask(q, k, 0.3, 0.6)
    want = attention(q, k, v, dout, m, rotary=r)
    with torch.autograd.graph.save_on_cpu():
        leaves = [x.detach().requires_grad_() for x in (q, k, v)]
        o = sparse_attention(*leaves, mask=m, checkpoint="int8", rotary=r)
    got = torch.autograd.grad(o, leaves, dout)
    assert torch.equal(o, want[0]) and all(torch.equal(a, c) for a, c in zip(got, want[1:]))


def test_fp32_gradients_through_the_binding():
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=600, d=128, seed=11, device="cuda")
    dout = synth.normal_like(q.shape, seed=12, device="cuda")
    s = b.Spa2(1, 2, 600, 128)
    m = s.block_mask(q, k, 0.2, 0.6)
    lse = torch.empty(1, 2, 600, device="cuda")
    o, packed = s.fwd_ckpt(q, k, v, m, lse=lse)
    o2, lse2 = s.fwd(q, k, v, m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a.data, c.data) for a, c in zip(packed, pack8(q, k, v)))
    grads = s.bwd_ckpt(packed, dout, m)
    s.check()
    dense = csr_to_dense(m.row_cnt.cpu().numpy(), m.row_idx.cpu().numpy(), s.Tn)
    want = oracle.masked_attn_bwd(*(kept(x)[2] for x in (q, k, v)), dense, f64(dout), 128, 64)
    for name, g, e in zip(("dQ", "dK", "dV"), grads, want):
        assert g.dtype == F32
        assert_close(g.double().cpu().numpy(), e, name)


def test_repeatable_and_safe_on_two_streams():
    """The same bits every time, also when two streams run the step at once."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=3, N=1500, d=64, seed=13, device="cuda")
    dout = synth.normal_like(q.shape, seed=14, device="cuda")
    m = block_mask(q, k, 0.2, 0.6)
    want = attention(q, k, v, dout, m)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(attention(q, k, v, dout, m))
    torch.cuda.synchronize()
    check_errors()
    for run in got:
        assert all(torch.equal(a, c) for a, c in zip(run, want))


def test_captured_steps():
    """Two captured steps, replayed at once on two streams on new inputs: each has workspaces of its own."""
    sets = []
    for i in range(2):
        q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=900, d=64, seed=20 + i, device="cuda")
        sets.append((q, k, v, synth.normal_like(q.shape, seed=30 + i, device="cuda"), block_mask(q, k, 0.3, 0.6)))
    attention(*sets[0])
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = attention(*s)
        graphs.append((g, out))
    for s in sets:
        s[0].copy_(torch.randn_like(s[0]))
    want = [attention(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for (g, _), st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    check_errors()
    for (_, out), w in zip(graphs, want):
        assert all(torch.equal(a, c) for a, c in zip(out, w))


# ---- the run of them together ---------------------------------------------------------
def test_rotary_mask_attention_and_checkpoints_together():
    """Projections -> rotary by grid positions -> mask -> attention on 8-bit checkpoints
    -> gradients of the projections. The turned q and k of apply_rotary go to the
    oracle; its dQ and dK, turned back in float64, bound the result: a turn mixes two
    elements, so the attention's error (2e-2 and half a bf16 step of its bf16
    gradient) grows by |cos| + |sin| <= 2^(1/2), and the turn rounds once more."""
    grid = (3, 8, 10)
    B, H, N, d = 1, 2, 240, 64
    x = synth.normal_like((B, N, 3, H, d), seed=40, device="cuda")
    q, k, v = (x[:, :, i].transpose(1, 2).detach().requires_grad_() for i in range(3))
    inv_freq, axes = axial_frequencies(d, device="cuda")
    r = Rotary(inv_freq, grid_positions(*grid, device="cuda"), axes=axes)
    dout = synth.normal_like((B, H, N, d), seed=41, device="cuda")
    o, cnt = sparse_attention(q, k, v, 0.4, 0.6, checkpoint="int8", rotary=r, return_mask=True)
    grads = torch.autograd.grad(o, (q, k, v), dout)
    check_errors()
    with torch.no_grad():
        qr, kr = apply_rotary(q, k, inv_freq=inv_freq, positions=r.positions, axes=axes)
    m = block_mask(qr, kr, 0.4, 0.6)
    assert torch.equal(m.row_cnt, cnt)
    dense = csr_to_dense(m.row_cnt.cpu().numpy(), m.row_idx.cpu().numpy(), m.row_idx.shape[-1])
    O, _ = oracle.masked_attn_fwd(f64(qr), f64(kr), f64(v), dense, 128, 64)
    assert_close_bf16_out(f64(o), O, "O")
    want = oracle.masked_attn_bwd(*(kept(t)[2] for t in (qr, kr, v)), dense, f64(dout), 128, 64)
    axis = np.repeat(np.arange(3), axes)
    angle = r.positions.cpu().numpy()[axis].T * inv_freq.cpu().numpy()
    c, s = np.cos(angle), np.sin(angle)
    for name, g, e in zip(("dQ", "dK"), grads, want):
        a, w = e[..., 0::2], e[..., 1::2]
        back = np.stack((a * c + w * s, w * c - a * s), -1).reshape(e.shape)
        within = 2 ** 0.5 * (2e-2 + np.repeat(np.maximum(bf16_half_ulp(a), bf16_half_ulp(w)), 2, -1)) + 1.01 * bf16_half_ulp(back)
        assert (np.abs(f64(g) - back) <= within).all(), name
    assert_close_bf16_out(f64(grads[2]), want[2], "dV")
    assert grads[0].transpose(1, 2).is_contiguous()   # in the order of the projection


def test_training_steps_run_on_checkpoints():
    """A block with projections, rotary and checkpointed attention: finite gradients of every weight over a few steps."""
    torch.manual_seed(0)
    B, N, H, d = 2, 600, 2, 64
    x = torch.randn(B, N, H * d, device="cuda")
    qkv = torch.nn.Linear(H * d, 3 * H * d, device="cuda")
    out = torch.nn.Linear(H * d, H * d, device="cuda")
    opt = torch.optim.SGD([*qkv.parameters(), *out.parameters()], lr=0.1)
    inv_freq, axes = axial_frequencies(d, device="cuda")
    r = Rotary(inv_freq, grid_positions(6, 10, 10, device="cuda"), axes=axes)
    for _ in range(3):
        q, k, v = (t.transpose(1, 2) for t in qkv(x).bfloat16().view(B, N, 3, H, d).unbind(2))
        o = sparse_attention(q, k, v, 0.1, 0.5, checkpoint="int8", rotary=r)
        loss = out(o.transpose(1, 2).reshape(B, N, H * d).float()).square().mean()
        opt.zero_grad()
        loss.backward()
        assert all(torch.isfinite(p.grad).all() and p.grad.any() for p in (*qkv.parameters(), *out.parameters()))
        opt.step()
    check_errors()
