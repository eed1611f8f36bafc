"""When the backward pass of a rotation may take over the packed arguments of the forward: not
where a saved tensor has come back with other strides or another type at the old address."""

import pytest
import torch

from trainable_block_sparse_pooled_b200 import binding as b
from trainable_block_sparse_pooled_b200 import rotary

F = torch.ones(4, dtype=torch.float64)


def spec(positions, axes=None, N=5):
    return rotary._spec(rotary.Rotary(F, positions, axes=axes), 2, N, 8, torch.device("cpu"))[0]


@pytest.mark.parametrize("shape,strides,axes", [
    ((3, 5), (7, 1), (2, 1, 1)), ((3, 5), (1, 3), (2, 1, 1)), ((2, 3, 5), (5, 10, 1), (2, 1, 1)), ((5,), (2,), None),
    ((2, 5), (0, 1), None), ((2, 5), (1, 2), None)])
def test_other_strides_at_the_same_address(shape, strides, axes):
    base = torch.arange(60)
    laid = base.as_strided(shape, strides)
    plain = base[:laid.numel()].view(shape)
    assert plain.data_ptr() == laid.data_ptr()
    assert b.rotary_spec_points(spec(laid, axes), F, laid) and b.rotary_spec_points(spec(plain, axes), F, plain)
    assert not b.rotary_spec_points(spec(laid, axes), F, plain)
    assert not b.rotary_spec_points(spec(plain, axes), F, laid)


def test_another_type_at_the_same_address():
    wide = torch.arange(5)
    narrow = wide.view(torch.int32)[:5]
    assert wide.data_ptr() == narrow.data_ptr()
    assert not b.rotary_spec_points(spec(wide), F, narrow) and not b.rotary_spec_points(spec(narrow), F, wide)
    assert not b.rotary_spec_points(spec(wide), F, None) and not b.rotary_spec_points(spec(None), F, wide)
    assert b.rotary_spec_points(spec(None), F, None)
