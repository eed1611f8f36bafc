"""What the checkpointed step's roundings leave of its gradients, against float64 at the kept values."""

import numpy as np
import pytest
import torch

import oracle
from tests._parity import csr_to_dense, f64
from trainable_block_sparse_pooled_b200 import binding as b
from trainable_block_sparse_pooled_b200 import synth
from trainable_block_sparse_pooled_b200.checkpoint import pack8, unpack8

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def gradients(q, k, v, dout, m, bq=b.BQ, bkv=b.BKV):
    """fp32 dQ, dK, dV of the kernels and their float64 values, at the kept values of q, k, v."""
    B, H, N, d = q.shape
    s = b.Spa2(B, H, N, d, bq=bq, bkv=bkv)
    packed = pack8(q, k, v)
    got = s.bwd_ckpt(packed, dout, m)
    s.check()
    dense = csr_to_dense(m.row_cnt.cpu().numpy(), m.row_idx.cpu().numpy(), m.row_idx.shape[-1])
    q8, k8, v8 = (f64(x) for x in unpack8(*packed))
    return [g.double().cpu().numpy() for g in got], oracle.masked_attn_bwd(q8, k8, v8, dense, f64(dout), bq, bkv)


def normal(N, d, H=1, seed=0):
    return [synth.normal_like((1, H, N, d), seed=seed + i, device="cuda") for i in range(4)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [8, 12, 16, 30, 60])
def test_queries_with_small_gradients_beside_large_ones(d, power):
    """Every fourth row of dO at 2^-power of the others. A row of dQ depends on its own row of dO alone, so it
    keeps its precision: relative to its norm it is off by the roundings of P, dP and dS, each
    relative to its term. P's exponent, up to 8 here, is a sum of d products in fp32: at most d * 2^-24 * 8 * ln 2
    = 4e-5 for d = 128; dP as much of its own sum of magnitudes; dS is a pair of fp16 (2^-22); the sum over 2000 keys in
    fp32 adds 2000 * 2^-24 = 1.2e-4 of its terms' magnitudes at worst. Errors of independent terms add up like the
    terms themselves, so the row's error stays below the sum of these, 3e-4 of its norm; 5e-4 leaves the rest."""
    q, k, v, dout = normal(2000, d, seed=power)
    dout[:, :, ::4] = torch.ldexp(dout[:, :, ::4].float(), torch.tensor(-power, device="cuda")).to(BF16)
    s = b.Spa2(1, 1, 2000, d)
    m = s.block_mask(q, k, 1.0, 1.0)
    got, want = gradients(q, k, v, dout, m)
    err = np.linalg.norm(got[0] - want[0], axis=-1) / np.linalg.norm(want[0], axis=-1)
    assert err.max() <= 5e-4, (power, err[..., ::4].max(), err[..., 1::4].max())


def test_keys_that_only_small_gradients_reach():
    """dK and dV are relative to the head's largest |dO|, brought into [4, 8): a dS below 2^-14 there is off by up to
    2^-25 (half of fp16's smallest step), a dO as much. The third query block has 2^-12 of the others' dO and keeps
    a key block that nobody else keeps: that block's dK and dV within those steps, and 2^-11 of each P and dS."""
    q, k, v, dout = normal(512, 64, seed=7)
    dout[0, 0, 256:384] *= 2.0 ** -12
    keep = torch.ones(1, 1, 4, 8, dtype=torch.bool)
    keep[..., 5] = False
    keep[0, 0, 2] = False
    keep[0, 0, 2, 5] = True

    def csr(x):
        n = x.shape[-1]
        ids = torch.where(x, torch.arange(n), n).sort(dim=-1).values.clamp(max=n - 1)
        return x.sum(-1).int().contiguous().cuda(), ids.int().contiguous().cuda()

    m = b.Mask(*csr(keep), *csr(keep.transpose(-1, -2)))
    got, want = gradients(q, k, v, dout, m)
    most = float(dout.float().abs().max())
    unit = 2.0 ** (np.floor(np.log2(most)) - 2)       # what dO is divided by
    rows, keys = slice(256, 384), slice(320, 384)
    q8, k8, v8 = (f64(x)[0, 0] for x in unpack8(*pack8(q, k, v)))
    do = f64(dout)[0, 0, rows]
    x = q8[rows] @ k8[keys].T / 8
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    dp = do @ v8[keys].T
    ds = p * (dp - (p * dp).sum(1, keepdims=True))
    # P, dP and D in fp32 are off by 64 additions of 2^-23 of magnitudes up to 8 (P's exponent), 2^-13 of their terms
    terms = p * (np.abs(do) @ np.abs(v8[keys]).T + np.abs(p * dp).sum(1, keepdims=True))
    lost = 2.0 ** -25 * unit                          # of a dS, or of an element of dO, below fp16's normal range
    off = lost + 2.0 ** -11 * np.abs(ds) + 2.0 ** -13 * terms + 2 * p * lost * np.abs(v8[keys]).sum(1).max()
    bound = (1 + 2.0 ** -13) * off.T @ np.abs(q8[rows]) / 8 + 2.0 ** -13 * (np.abs(ds).T @ np.abs(q8[rows])) / 8
    assert (np.abs(got[1][0, 0, keys] - want[1][0, 0, keys]) <= bound).all()
    bound = p.sum(0)[:, None] * lost + 2.0 ** -10 * (p.T @ np.abs(do)) + 2.0 ** -25 * np.abs(do).sum(0)
    assert (np.abs(got[2][0, 0, keys] - want[2][0, 0, keys]) <= bound).all()


@pytest.mark.parametrize("N,d,bq,bkv", [(1000, 128, 128, 64), (1000, 64, 64, 128), (130, 128, 256, 64), (2049, 128, 128, 64)])
def test_query_gradients_among_sink_keys(N, d, bq, bkv):
    """Sink keys of eight times the norm, whose terms cancel in dQ: the pass carries dS as a pair, as the plain backward
    does, and stays within a tenth of the 2e-2 that is promised. One half of 11 bits is off by up to 2^-12 |dS| |K| for
    each sink, with |dS| to 8 and |K| to 50 times the scale 1e-2 and more; of the pair 2^-22 is left, and P, dP and D
    in fp32: a relative 16 * 2^-23 * 24 (the exponent, P and LSE) = 5e-5 of those terms, 1e-3 of 8 * 50 * 0.1 / 2."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=N, d=d, seed=N + d, device="cuda")
    dout = synth.normal_like(q.shape, seed=N, device="cuda")
    s = b.Spa2(1, 2, N, d, bq=bq, bkv=bkv)
    got, want = gradients(q, k, v, dout, s.block_mask(q, k, 0.2, 0.6), bq, bkv)
    assert np.abs(got[0] - want[0]).max() <= 2e-3


@pytest.mark.parametrize("power", [-115, -100, 100, 115])
def test_gradients_of_any_size_that_bf16_holds(power):
    """Powers of two of dO's head come through, also near the ends of bf16's range. The elements of dO are whole
    numbers up to 8, so that 2^-115 of them is exact in bf16 (its smallest normal number is 2^-126);
    the results are compared in fp32, whose own steps below 2^-126 are 2^-149."""
    q, k, v, dout = normal(300, 64, H=2, seed=3)
    dout = dout.float().round().clamp(-8, 8).to(BF16)
    s = b.Spa2(1, 2, 300, 64)
    m = s.block_mask(q, k, 0.5, 0.5)
    packed = pack8(q, k, v)
    want = s.bwd_ckpt(packed, dout, m)
    s.check()
    by = torch.tensor(power, device="cuda")
    got = s.bwd_ckpt(packed, torch.ldexp(dout.double(), by).to(BF16), m)
    s.check()
    for g, w in zip(got, want):
        assert ((g.double() - torch.ldexp(w.double(), by)).abs() <= 2.0 ** -149).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [4, 8, 10])
def test_small_values(d, power):
    """V at 2^-power: dQ and dK are 2^-power of what they were, dV is the same, bit for bit. dP is exact in dO's and
    V's powers of two, and dO is taken up by as much as V has gone down (2^12 in all, of which |V| of 4 to 8
    takes 1 or 2), so dS is rounded as before. dO in whole numbers, which fp16 holds however they are scaled."""
    q, k, v, dout = normal(2000, d, seed=power)
    dout = (2 * dout.float()).round().to(BF16)
    assert 4 <= v.abs().max() < 8
    s = b.Spa2(1, 1, 2000, d)
    m = s.block_mask(q, k, 1.0, 1.0)
    want = s.bwd_ckpt(pack8(q, k, v), dout, m)
    by = torch.tensor(-power, device="cuda")
    got = s.bwd_ckpt(pack8(q, k, torch.ldexp(v.float(), by).to(BF16)), dout, m)
    s.check()
    assert torch.equal(got[0], torch.ldexp(want[0], by)) and torch.equal(got[1], torch.ldexp(want[1], by))
    assert torch.equal(got[2], want[2])
