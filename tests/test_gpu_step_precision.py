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
