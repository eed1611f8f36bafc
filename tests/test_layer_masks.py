"""Block masks whose lists change between the two passes of the checkpointed attention, without a GPU."""

import pytest
import torch

from trainable_block_sparse_pooled_b200 import autograd, binding as b
from trainable_block_sparse_pooled_b200.checkpoint import Packed


class Workspace(b.Spa2):
    """A Spa2 whose kernels do nothing but hand back what they were given."""

    def __init__(self):
        super().__init__(1, 1, 128, 64, device=torch.device("cpu"), lazy=True)
        self.watch = autograd._NoWatch()

    def fwd_ckpt(self, q, k, v, mask, scale=0.0):
        return q.clone(), Packed.several_like(q, 3)

    def bwd_ckpt(self, kept, do, mask, scale=0.0, grad_dtype=None):
        self.used = mask
        return do, do, do


@pytest.fixture
def step(monkeypatch):
    s = Workspace()
    monkeypatch.setattr(autograd, "_spa", lambda *a, **kw: s)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    def run(mask, between=lambda: None):
        q = torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16, requires_grad=True)
        o = autograd.CheckpointedAttentionFunction.apply(q, q, q, 0.0, mask, b.BQ, b.BKV)
        between()
        o.sum().backward()
        return s.used
    return run


def lists():
    i = lambda *s: torch.ones(*s, dtype=torch.int32)  # noqa: E731
    return [i(1, 1, 1), i(1, 1, 1, 2), i(1, 1, 2), i(1, 1, 2, 1)]


@pytest.mark.parametrize("n", range(4))
def test_a_list_written_in_place_is_noticed(step, n):
    m = b.Mask(*lists())
    with pytest.raises(RuntimeError, match="mask"):
        step(m, lambda: (m.row_cnt, m.row_idx, m.col_cnt, m.col_idx)[n].zero_())


def test_other_lists_put_into_the_mask_are_not_used(step):
    first, m = lists(), b.Mask(*lists())
    m.row_cnt, m.row_idx, m.col_cnt, m.col_idx = first
    used = step(m, lambda: m.__dict__.update(b.Mask(*lists()).__dict__))
    assert used.row_cnt is first[0] and used.row_idx is first[1] and used.col_cnt is first[2] and used.col_idx is first[3]


def test_masks_may_be_read_and_used_again_and_come_from_inference_mode(step):
    m = b.Mask(*lists())
    for _ in range(2):
        step(m, lambda: m.kept_blocks())
    with torch.inference_mode():
        frozen = b.Mask(*lists())
    step(frozen)


def test_a_mask_built_into_given_buffers_counts_as_written(monkeypatch):
    """The kernels write by address: the call itself tells torch."""
    s = b.Spa2(1, 1, 128, 64, device=torch.device("cpu"), lazy=True)
    monkeypatch.setattr(b, "spa2_block_mask", lambda *a: b.OK)
    monkeypatch.setattr(b, "_stream", lambda t: 0)
    q = torch.zeros(1, 1, 128, 64, dtype=torch.bfloat16)
    m = s.block_mask(q, q, 0.5, 0.5)
    before = m.versions()
    assert s.block_mask(q, q, 0.5, 0.5, mask=m) is m and all(v > w for v, w in zip(m.versions(), before))
    with torch.inference_mode():
        frozen = s.block_mask(q, q, 0.5, 0.5)
        s.block_mask(q, q, 0.5, 0.5, mask=frozen)
    s.block_mask(q, q, 0.5, 0.5, mask=frozen)
