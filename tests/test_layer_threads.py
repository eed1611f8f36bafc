"""Host threads that share a workspace, without a GPU: the launches of one operation, and
the copy of its status, are not interrupted by another thread's."""

import threading
import time

import pytest
import torch

from trainable_block_sparse_pooled_b200 import autograd, binding as b


class Workspace(b.Spa2):
    """A Spa2 whose calls take a moment, as a C call that has released the interpreter does, and record who is in."""

    def __init__(self):
        super().__init__(1, 1, 128, 64, device=torch.device("cpu"), lazy=True)
        self.inside, self.overlaps, self.calls = 0, 0, 0
        self.watch = self

    def _call(self):
        self.inside += 1
        self.overlaps += self.inside > 1
        self.calls += 1
        time.sleep(0.002)

    def poll(self):
        pass

    def after(self, ops):     # the status copy ends an operation
        time.sleep(0.001)
        self.inside -= 1

    def block_mask(self, q, k, k_frac, p_frac, mask=None):
        self._call()
        i = lambda *s: torch.ones(*s, dtype=torch.int32)  # noqa: E731
        return b.Mask(i(1, 1, 1), i(1, 1, 1, 2), i(1, 1, 2), i(1, 1, 2, 1))

    def fwd(self, q, *args, **kw):
        self._call()
        self.o_lo = torch.full_like(q, float(threading.get_ident() % 97))
        return q.clone(), q.new_zeros(1, 1, 128, dtype=torch.float32)

    def bwd(self, q, k, v, o, lse, do, mask, scale, o_lo=None, grad_dtype=None):
        self._call()
        assert (o_lo == o_lo.flatten()[0]).all() and o_lo.flatten()[0] == q.flatten()[0]
        return do, do, do

    def fwd_ckpt(self, q, *args, **kw):
        self._call()
        return q.clone(), b_packed(q)

    def bwd_ckpt(self, kept, do, *args, **kw):
        self._call()
        return do, do, do


def b_packed(q):
    from trainable_block_sparse_pooled_b200.checkpoint import Packed
    return Packed.several_like(q, 3)


@pytest.mark.parametrize("checkpoint", [False, True])
def test_operations_on_one_workspace_do_not_interleave(monkeypatch, checkpoint):
    s = Workspace()
    monkeypatch.setattr(autograd, "_spa", lambda *a, **kw: s)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    failed = []

    def work():
        try:
            me = float(threading.get_ident() % 97)
            for _ in range(5):
                q = torch.full((1, 1, 128, 64), me, dtype=torch.bfloat16, requires_grad=True)
                m = autograd.block_mask(q.detach(), q.detach(), 0.5, 0.5)
                if checkpoint:
                    o = autograd.CheckpointedAttentionFunction.apply(q, q, q, 0.0, m, b.BQ, b.BKV)
                else:
                    o, _ = autograd.SparseAttentionFunction.apply(q, q, q, 0.0, 0.0, 0.0, m, b.BQ, b.BKV)
                o.sum().backward()
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and s.calls == 45 and s.overlaps == 0 and s.inside == 0


def test_one_workspace_set_per_shape_and_stream(monkeypatch):
    """Threads that ask for the first time at once get the same set."""
    made = []

    class Slow(b.Spa2):
        def __init__(self, *args, **kw):
            time.sleep(0.02)
            made.append(self)

    class Watch:
        def __init__(self, spa):
            pass

        def poll(self):
            pass

    monkeypatch.setattr(autograd.b, "Spa2", Slow)
    monkeypatch.setattr(autograd, "_StatusWatch", Watch)
    monkeypatch.setattr(autograd, "_cache", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    got = []
    threads = [threading.Thread(target=lambda: got.append(autograd._spa(1, 1, 128, 64, torch.device("cuda:0"))))
               for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and len(got) == 4 and all(s is made[0] for s in got)
