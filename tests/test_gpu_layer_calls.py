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


# ---- forward mode and tracing ---------------------------------------------------------
@pytest.mark.parametrize("wanted", [False, True])
def test_forward_mode_derivatives_of_rotary(wanted):
    """The map is linear: the tangent is turned as its tensor is, bit for bit."""
    f = rotary_frequencies(32, device="cuda")[0]
    q, tq, k = (torch.randn(2, 3, 21, 64, device="cuda") for _ in range(3))
    pos = torch.arange(21, device="cuda") * 3
    kw = dict(inv_freq=f, positions=pos, layout="half", scale=1.25)
    want = apply_rotary(tq, **kw)
    with fwd_ad.dual_level():
        dual = fwd_ad.make_dual(q.requires_grad_(wanted), tq)
        y = fwd_ad.unpack_dual(apply_rotary(dual, **kw))
        assert y.tangent is not None and torch.equal(y.tangent, want)
        assert torch.equal(y.primal, apply_rotary(q.detach(), **kw))
        yq, yk = (fwd_ad.unpack_dual(x) for x in apply_rotary(dual, k, **kw))
        assert torch.equal(yq.tangent, want) and (yk.tangent is None or not yk.tangent.any())
        yk, yq = (fwd_ad.unpack_dual(x) for x in apply_rotary(k, dual, **kw))
        assert torch.equal(yq.tangent, want) and (yk.tangent is None or not yk.tangent.any())


def test_reverse_over_forward_mode_of_rotary():
    f = rotary_frequencies(64, device="cuda")[0]
    q, t, h = (torch.randn(1, 2, 9, 64, device="cuda") for _ in range(3))
    t.requires_grad_()
    with fwd_ad.dual_level():
        tangent = fwd_ad.unpack_dual(apply_rotary(fwd_ad.make_dual(q, t), inv_freq=f)).tangent
        (got,) = torch.autograd.grad(tangent, t, h)
    leaf = q.detach().requires_grad_()
    assert torch.equal(got, torch.autograd.grad(apply_rotary(leaf, inv_freq=f), leaf, h)[0])


@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_forward_mode_through_the_attention_is_refused(checkpoint):
    """The attention has no forward-mode derivative: with rotary in front as without it, the call raises."""
    q, k, v, _ = problem()
    m = block_mask(q, k, 0.3, 0.6)
    r = Rotary(rotary_frequencies(64, device="cuda")[0])
    for i in range(3):
        for rotary in (None, r):
            with fwd_ad.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
                xs = [q, k, v]
                xs[i] = fwd_ad.make_dual(xs[i], torch.ones_like(q))
                sparse_attention(*xs, mask=m, rotary=rotary, checkpoint=checkpoint)


def test_checkpoints_refuse_forward_mode():
    x = torch.randn(4, 64, device="cuda")
    with fwd_ad.dual_level(), pytest.raises(RuntimeError):
        pack8(fwd_ad.make_dual(x, torch.ones_like(x)))


def test_traced_rotary_follows_its_inputs():
    f = rotary_frequencies(64, device="cuda")[0]
    q, pos = torch.randn(1, 2, 9, 64, device="cuda"), torch.arange(9, device="cuda")
    traced = torch.jit.trace(lambda x, p: apply_rotary(x, inv_freq=f, positions=p), (q, pos))
    q2, pos2, h = torch.randn_like(q).requires_grad_(), pos * 7 + 1, torch.randn_like(q)
    want = apply_rotary(q2, inv_freq=f, positions=pos2)
    got = traced(q2, pos2)
    assert torch.equal(got, want)
    assert torch.equal(torch.autograd.grad(got, q2, h)[0], torch.autograd.grad(want, q2, h)[0])


def test_traced_checkpoints_are_refused():
    """A trace would hold the buffers, not what fills them."""
    x = torch.randn(4, 64, device="cuda")
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda t: unpack8(*pack8(t))[0], (x,))
    kept = pack8(x)
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda t: unpack8(*kept)[0] + t, (x,))
    q, k, v, _ = problem()
    with pytest.raises(RuntimeError):   # its mask would be that of the traced inputs
        torch.jit.trace(lambda *xs: sparse_attention(*xs, 0.3, 0.6, checkpoint="int8"),
                        tuple(t.requires_grad_() for t in (q, k, v)))


# ---- streams and threads --------------------------------------------------------------
def test_many_calls_ahead_wait_for_their_own_stream_alone():
    """Forty calls while another stream is busy for much longer: the calls return, and
    check_errors too, before that stream is done."""
    q, k, v, _ = problem(N=256)
    m = block_mask(q, k, 0.3, 0.6)
    sparse_attention(q, k, v, mask=m)
    check_errors()
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(6_000_000_000)     # about three seconds
        busy.record()
    torch.cuda._sleep(200_000_000)           # a tenth of a second: the status copies are behind it
    for _ in range(40):
        sparse_attention(q, k, v, mask=m)
    assert not busy.query()
    check_errors()
    assert not busy.query()
    torch.cuda.synchronize()


def test_errors_are_reported_while_another_stream_is_busy():
    q, k, v, _ = problem(N=256)
    m = block_mask(q, k, 1.0, 1.0)
    check_errors()
    bad = v.clone()
    bad[0, 0, 3, 3] = 1e6
    side, busy = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(6_000_000_000)
        busy.record()
    sparse_attention(q, k, bad, mask=m)
    with pytest.raises(b.Spa2Error) as e:
        check_errors()
    assert e.value.code == b.ERR_RANGE and not busy.query()
    torch.cuda.synchronize()
    sparse_attention(q, k, v, mask=m)
    check_errors()


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


# ---- masks that are filled again ------------------------------------------------------
@pytest.mark.parametrize("how", ["block_mask", "in place"])
def test_a_mask_changed_before_the_backward_pass_is_noticed(how):
    """The gradients are those of the attention under the mask's lists as they are in the backward pass: not of the
    o that was returned, if they are others by then."""
    q, k, v, dout = problem()
    s = b.Spa2(1, 2, 500, 64)
    m = s.block_mask(q, k, 0.2, 0.4)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = sparse_attention(*leaves, mask=m, checkpoint="int8")
    if how == "block_mask":
        s.block_mask(k, q, 0.5, 0.9, mask=m)
    else:
        m.col_cnt.fill_(1)
    with pytest.raises(RuntimeError, match="mask"):
        torch.autograd.grad(o, leaves, dout)


def test_other_lists_put_into_a_mask_do_not_reach_the_backward_pass():
    q, k, v, dout = problem()
    m, other = block_mask(q, k, 0.2, 0.4), block_mask(q, k, 0.6, 0.9)
    want = step(q, k, v, dout, b.Mask(m.row_cnt, m.row_idx, m.col_cnt, m.col_idx))
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = sparse_attention(*leaves, mask=m, checkpoint="int8")
    m.row_cnt, m.row_idx, m.col_cnt, m.col_idx = other.row_cnt, other.row_idx, other.col_cnt, other.col_idx
    assert all(torch.equal(a, w) for a, w in zip(torch.autograd.grad(o, leaves, dout), want[1:]))


def test_a_mask_built_in_inference_mode_serves_a_training_step():
    q, k, v, dout = problem()
    with torch.inference_mode():
        frozen = block_mask(q, k, 0.2, 0.6)
    want = step(q, k, v, dout, block_mask(q, k, 0.2, 0.6))
    assert all(torch.equal(a, w) for a, w in zip(step(q, k, v, dout, frozen), want))


# ---- C entry points -------------------------------------------------------------------
def test_rotary_through_the_binding():
    """spa2_rotary with its structures: rows of a wider buffer turned into another, nothing beside them written."""
    f = rotary_frequencies(32, device="cuda")[0]
    x = torch.randn(2, 3, 21, 40, device="cuda").to(BF16)
    y = torch.full((2, 3, 21, 40), 55.0, device="cuda").to(BF16)
    t = b.spa2_rotary_tensor(x.data_ptr(), y.data_ptr(), 3)
    t.x_stride[:] = t.y_stride[:] = x.stride()[:3]
    s = b.spa2_rotary_spec()
    s.axes, s.inv_freq, s.rotary_dim, s.layout, s.scale = 1, f.data_ptr(), 32, b.ROTARY_HALF, 1.5
    s.pairs[0] = 16
    stream = torch.cuda.current_stream().cuda_stream
    for inverse in (False, True):
        assert b.spa2_rotary((b.spa2_rotary_tensor * 1)(t), 2, 21, 36, b.DTYPE_BF16, s, inverse, stream) == b.OK
        leaf = x[..., :36].detach().requires_grad_()
        out = apply_rotary(leaf, inv_freq=f, layout="half", scale=1.5)
        want = torch.autograd.grad(out, leaf, leaf.detach())[0] if inverse else out.detach()
        assert torch.equal(y[..., :36], want) and (y[..., 36:] == 55.0).all()
