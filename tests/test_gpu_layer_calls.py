"""Calls around the attention layer that a training program makes in unusual ways:
forward-mode derivatives, traced modules, saved tensors on the host, two host threads
on one stream, work on other streams, masks that are filled again."""

import threading

import pytest
import torch
import torch.autograd.forward_ad as fwd_ad

from trainable_block_sparse_pooled_b200 import binding as b
from trainable_block_sparse_pooled_b200 import synth
from trainable_block_sparse_pooled_b200.autograd import block_mask, check_errors, sparse_attention
from trainable_block_sparse_pooled_b200.checkpoint import pack8, unpack8
from trainable_block_sparse_pooled_b200.rotary import Rotary, apply_rotary, axial_frequencies, grid_positions, rotary_frequencies

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def problem(B=1, H=2, N=500, d=64, seed=1):
    q, k, v = synth.gaussian_with_sinks(B=B, H=H, N=N, d=d, seed=seed, device="cuda")
    return q, k, v, synth.normal_like(q.shape, seed=seed + 100, device="cuda")


def step(q, k, v, dout, mask, **kw):
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = sparse_attention(*leaves, mask=mask, checkpoint="int8", **kw)
    return (o.detach(), *torch.autograd.grad(o, leaves, dout))


# ---- saved tensors that come back with other strides ----------------------------------
def test_positions_that_only_the_graph_holds_come_back_contiguous():
    """A slice of grid positions (height and width 250 apart in memory, 200 tokens used), offloaded: save_on_cpu
    returns it contiguous, and the allocator may give it the block that the slice had."""
    q = torch.randn(1, 2, 200, 64, device="cuda")
    h = torch.randn_like(q)
    inv_freq, axes = axial_frequencies(64, device="cuda")
    leaf = q.detach().requires_grad_()
    want = torch.autograd.grad(apply_rotary(leaf, inv_freq=inv_freq, axes=axes,
                                            positions=grid_positions(5, 5, 10, device="cuda")[:, :200]), leaf, h)[0]
    for pin in (False, True):
        leaf = q.detach().requires_grad_()
        with torch.autograd.graph.save_on_cpu(pin_memory=pin):
            y = apply_rotary(leaf, inv_freq=inv_freq, axes=axes, positions=grid_positions(5, 5, 10, device="cuda")[:, :200])
        assert torch.equal(torch.autograd.grad(y, leaf, h)[0], want)


def test_two_threads_on_one_stream():
    """The same shape from two host threads, both on the default stream, each with tensors of its own: each gets
    what it gets alone."""
    sets = [problem(seed=50 + i, N=700) for i in range(2)]
    masks = [block_mask(s[0], s[1], 0.3, 0.6) for s in sets]

    def both(s, m):
        q, k, v, dout = s
        out = list(step(q, k, v, dout, m))
        leaves = [x.detach().requires_grad_() for x in (q, k, v)]
        o = sparse_attention(*leaves, mask=m)
        return out + [o.detach(), *torch.autograd.grad(o, leaves, dout)]

    want = [both(s, m) for s, m in zip(sets, masks)]
    right = [0, 0]

    def work(i):
        for _ in range(60):
            right[i] += all(torch.equal(a, w) for a, w in zip(both(sets[i], masks[i]), want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    check_errors()
    assert right == [60, 60]
