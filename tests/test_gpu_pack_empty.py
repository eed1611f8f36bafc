"""Empty tensors among others that pack8 and unpack8 take in one launch."""

import pytest
import torch

from trainable_block_sparse_pooled_b200 import binding as b
from trainable_block_sparse_pooled_b200.checkpoint import pack8, unpack8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_empty_tensors_beside_ragged_rows(dtype):
    """Rows of whole chunks but not of whole groups (40 = 32 + 8), beside tensors without rows: each comes back as
    it does alone, and the empty ones empty, wherever they stand."""
    x = torch.randn(7, 40, device="cuda").to(dtype)
    y = torch.randn(33, 72, device="cuda").to(dtype)
    empty = [torch.empty(shape, device="cuda", dtype=dtype) for shape in ((0, 64), (0, 40), (3, 0, 8))]
    alone = [unpack8(*pack8(t))[0] for t in (x, y)]
    for xs in ([empty[0], x, empty[1], y, empty[2]], [x, empty[0], y], [empty[2], empty[1], y, x]):
        back = unpack8(*pack8(*xs))
        assert [t.shape for t in back] == [t.shape for t in xs]
        full = [t for t in back if t.numel()]
        want = alone if any(t is x for t in xs[:2]) else alone[::-1]
        assert all(torch.equal(a, w) for a, w in zip(full, want))
    assert all(t.numel() == 0 for t in unpack8(*pack8(*empty)))


def test_empty_tensors_need_no_buffers():
    """rows = 0 with null pointers, between two others: nothing of it is read."""
    x = torch.randn(2, 5, 40, device="cuda").to(torch.bfloat16)
    codes = torch.zeros(2, 200, dtype=torch.int8, device="cuda")
    exps = torch.zeros(2, 10, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(x)
    stream = torch.cuda.current_stream().cuda_stream
    for call, t in ((b.spa2_pack8, x), (b.spa2_unpack8, out)):
        item = lambda i: b.spa2_pack8_tensor(t[i].data_ptr(), codes[i].data_ptr(), exps[i].data_ptr(), 5, 40)  # noqa: E731
        items = (b.spa2_pack8_tensor * 3)(item(0), b.spa2_pack8_tensor(None, None, None, 0, 40), item(1))
        assert call(items, b.DTYPE_BF16, stream) == b.OK
    assert torch.equal(out, torch.stack(unpack8(*pack8(x[0], x[1]))))
