"""Refusals of the 8-bit checkpoints that need no GPU: inside a trace they say so, whatever the tensors are."""

import pytest
import torch

from trainable_block_sparse_pooled_b200 import autograd, checkpoint


def test_traces_are_refused():
    x = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16)
    kept = checkpoint.Packed.empty_like(x)
    for call in (lambda t: checkpoint.pack8(t), lambda t: checkpoint.unpack8(kept)[0] + t,
                 lambda t: autograd.sparse_attention(t, t, t, 0.5, 0.5, checkpoint="int8")):
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(call, (x,))
