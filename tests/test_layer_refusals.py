"""Refusals of the layer's calls that need no GPU."""

import pytest
import torch

from trainable_block_sparse_pooled_b200 import autograd, checkpoint, rotary


def test_traces_are_refused():
    x = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16)
    kept = checkpoint.Packed.empty_like(x)
    for call in (lambda t: checkpoint.pack8(t), lambda t: checkpoint.unpack8(kept)[0] + t,
                 lambda t: autograd.sparse_attention(t, t, t, 0.5, 0.5, checkpoint="int8")):
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(call, (x,))


def test_a_scale_that_wants_a_gradient_is_refused():
    """It would be taken as a number, and its gradient lost."""
    q, f = torch.zeros(1, 1, 4, 8), torch.ones(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="scale"):
        rotary.apply_rotary(q, inv_freq=f, scale=torch.ones((), requires_grad=True))
