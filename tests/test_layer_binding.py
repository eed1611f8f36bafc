"""Spa2's calls on checkpoints hand addresses to the kernels: shapes and layouts that do not
fit are refused first."""

import pytest
import torch

from trainable_block_sparse_pooled_b200 import binding as b
from trainable_block_sparse_pooled_b200.checkpoint import Packed

BF16 = torch.bfloat16


@pytest.fixture
def spa(monkeypatch):
    def launched(*args):
        raise AssertionError("a call of the library")

    monkeypatch.setattr(b, "spa2_sparse_attn_fwd_ckpt", launched)
    monkeypatch.setattr(b, "spa2_sparse_attn_bwd_ckpt", launched)
    return b.Spa2(1, 2, 128, 64, device=torch.device("cpu"), lazy=True)


MASK = b.Mask(*(torch.ones(n, dtype=torch.int32) for n in (2, 4, 4, 4)))
GOOD = torch.zeros(1, 2, 128, 64, dtype=BF16)
BAD = [GOOD[:, :1], GOOD[:, :, :64], GOOD.float(), torch.zeros(1, 128, 2, 64, dtype=BF16).transpose(1, 2),
       torch.zeros(2, 1, 128, 64, dtype=BF16), GOOD.half()]


@pytest.mark.parametrize("bad", BAD)
def test_forward_refusals(spa, bad):
    for i in range(3):
        xs = [GOOD, GOOD, GOOD]
        xs[i] = bad
        with pytest.raises(ValueError):
            spa.fwd_ckpt(*xs, MASK)


@pytest.mark.parametrize("bad", BAD)
def test_backward_refusals(spa, bad):
    with pytest.raises(ValueError):
        spa.bwd_ckpt(Packed.several_like(GOOD, 3), bad, MASK)


def test_checkpoints_of_other_shapes_are_refused(spa):
    good, small = Packed.empty_like(GOOD), Packed.empty_like(GOOD[:, :, :64])
    for kept in ((good, good), (small, good, good), (good, small, good), (good, good, small), (good,) * 4):
        with pytest.raises(ValueError):
            spa.bwd_ckpt(kept, GOOD, MASK)
