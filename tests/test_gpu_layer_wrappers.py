"""The layer's calls inside what torch offers around them: recomputation, graphed callables,
captured steps that build their own mask, saved tensors in pinned memory."""

import pytest
import torch
import torch.utils.checkpoint

from trainable_block_sparse_pooled_b200 import synth
from trainable_block_sparse_pooled_b200.autograd import check_errors, sparse_attention
from trainable_block_sparse_pooled_b200.checkpoint import pack8, unpack8
from trainable_block_sparse_pooled_b200.rotary import Rotary, apply_rotary, axial_frequencies, grid_positions, rotary_frequencies

pytestmark = pytest.mark.gpu


@pytest.fixture
def layer():
    """(step, q, k, v, dout): rotary by grid positions, a mask of its own and 8-bit checkpoints."""
    q, k, v = synth.gaussian_with_sinks(B=1, H=2, N=600, d=64, seed=3, device="cuda")
    inv_freq, axes = axial_frequencies(64, device="cuda")
    r = Rotary(inv_freq, grid_positions(6, 10, 10, device="cuda"), axes=axes)

    def run(q, k, v):
        return sparse_attention(q, k, v, 0.2, 0.6, checkpoint="int8", rotary=r)

    yield run, q, k, v, synth.normal_like(q.shape, seed=4, device="cuda")
    check_errors()


def gradients(run, q, k, v, dout):
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = run(*leaves)
    return (o.detach(), *torch.autograd.grad(o, leaves, dout))


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_in_the_backward_pass(layer, reentrant):
    run, q, k, v, dout = layer
    want = gradients(run, q, k, v, dout)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = torch.utils.checkpoint.checkpoint(run, *leaves, use_reentrant=reentrant)
    o.backward(dout)
    assert torch.equal(o, want[0]) and all(torch.equal(x.grad, w) for x, w in zip(leaves, want[1:]))


def test_saved_tensors_in_pinned_memory(layer):
    run, q, k, v, dout = layer
    want = gradients(run, q, k, v, dout)
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    with torch.autograd.graph.save_on_cpu(pin_memory=True):
        o = run(*leaves)
    assert all(torch.equal(a, w) for a, w in zip(torch.autograd.grad(o, leaves, dout), want[1:]))


def test_captured_with_a_mask_of_its_own(layer):
    """Replayed on other inputs, the graph builds their mask."""
    run, q, k, v, dout = layer
    gradients(run, q, k, v, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients(run, q, k, v, dout)
    q2, k2, v2 = synth.gaussian_with_sinks(B=1, H=2, N=600, d=64, seed=5, device="cuda")
    for a, c in zip((q, k, v), (q2, k2, v2)):
        a.copy_(c)
    want = gradients(run, q, k, v, dout)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(out, want))


def test_graphed_callable(layer):
    """Forward and backward captured apart, as torch.cuda.make_graphed_callables does."""
    run, q, k, v, dout = layer
    samples = tuple(x.clone().requires_grad_() for x in (q, k, v))
    graphed = torch.cuda.make_graphed_callables(run, samples)
    q2, k2, v2 = synth.gaussian_with_sinks(B=1, H=2, N=600, d=64, seed=6, device="cuda")
    for xs in ((q, k, v), (q2, k2, v2), (q, k, v)):
        want = gradients(run, *xs, dout)
        leaves = [x.detach().requires_grad_() for x in xs]
        o = graphed(*leaves)
        got = torch.autograd.grad(o, leaves, dout)
        assert torch.equal(o, want[0]) and all(torch.equal(a, w) for a, w in zip(got, want[1:]))


def test_kept_graph_gives_the_same_gradients_again(layer):
    run, q, k, v, dout = layer
    leaves = [x.detach().requires_grad_() for x in (q, k, v)]
    o = run(*leaves)
    first = torch.autograd.grad(o, leaves, dout, retain_graph=True)
    for x in leaves:
        x.data.zero_()        # the 8-bit values are what counts
    assert all(torch.equal(a, w) for a, w in zip(torch.autograd.grad(o, leaves, dout), first))


def test_some_of_the_inputs_want_gradients(layer):
    run, q, k, v, dout = layer
    want = gradients(run, q, k, v, dout)[1:]
    for i in range(3):
        xs = [x.detach().clone() for x in (q, k, v)]
        xs[i].requires_grad_()
        assert torch.equal(torch.autograd.grad(run(*xs), xs[i], dout)[0], want[i])


def test_one_tensor_for_all_three(layer):
    run, q, _, _, dout = layer
    x = q.detach().requires_grad_()
    want = gradients(run, q, q, q, dout)[1:]
    got = torch.autograd.grad(run(x, x, x), x, dout)[0]
    # three bf16 gradients added up in bf16, in the order of their arrival: half a step of each sum, 2^-8 of it
    total = sum(w.double() for w in want)
    assert ((got.double() - total).abs() <= 2 * 2.0 ** -8 * (sum(w.double().abs() for w in want))).all()


def test_function_transforms_are_refused(layer):
    """torch.func has no rule for these calls, and hands them tensors without memory: they raise, and do not run past
    the transform."""
    run, q, k, v, _ = layer
    f = rotary_frequencies(64, device="cuda")[0]
    x = torch.randn(2, 1, 2, 8, 64, device="cuda")
    for call in (lambda t: apply_rotary(t, inv_freq=f), lambda t: unpack8(*pack8(t))[0]):
        with pytest.raises(RuntimeError):
            torch.func.jvp(call, (x[0],), (torch.ones_like(x[0]),))
        with pytest.raises(RuntimeError):
            torch.func.grad(lambda t: call(t).sum())(x[0])
        with pytest.raises(RuntimeError):
            torch.func.vmap(call)(x)
        with pytest.raises(RuntimeError):
            torch.func.vmap(call, in_dims=4)(x.movedim(0, 4))
    with pytest.raises(RuntimeError):
        torch.func.jvp(run, (q, k, v), (torch.ones_like(q),) * 3)
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda t: run(t, k, v).float().sum())(q)
