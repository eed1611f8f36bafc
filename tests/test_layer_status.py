"""The ring of status copies without a GPU: what is waited for when it is full, when it is
drained and when it holds an error. Copies land when the test lets them."""

import ctypes
import threading
from types import SimpleNamespace

import pytest
import torch

from trainable_block_sparse_pooled_b200 import autograd, binding as b


class Ring:
    """A _StatusWatch over ordinary memory, whose copies are made by `land`."""

    def __init__(self, monkeypatch):
        monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: t)
        monkeypatch.setattr(b, "_stream", lambda t: 0)
        monkeypatch.setattr(b, "spa2_status_fetch", lambda ws, host, stream: self.queue.append((ws, host)) or b.OK)

        def synchronize(device=None):
            raise AssertionError("waits for the whole device")

        monkeypatch.setattr(torch.cuda, "synchronize", synchronize)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)   # no query without a GPU
        self.queue, self.status = [], torch.zeros(5, dtype=torch.int32)
        ws = [SimpleNamespace(data_ptr=lambda i=i: i) for i in range(5)]
        self.watch = autograd._StatusWatch(SimpleNamespace(ws=ws, device=torch.device("cuda:0")))

    def land(self, n=1, code=b.OK):
        for _ in range(n):
            _, host = self.queue.pop(0)
            ctypes.c_int32.from_address(host).value = code


@pytest.fixture
def ring(monkeypatch):
    return Ring(monkeypatch)


def later(call, *args):
    t = threading.Timer(0.05, call, args)
    t.start()
    return t


def test_a_full_ring_waits_for_its_oldest_copy_alone(ring):
    for _ in range(16):
        ring.watch.after((b.OP_FWD,))
    later(ring.land)
    ring.watch.after((b.OP_FWD,))
    assert len(ring.watch.pending) == 16 and len(ring.queue) == 16


def test_draining_waits_for_each_copy(ring):
    for _ in range(3):
        ring.watch.after((b.OP_MASK, b.OP_FWD))
    later(ring.land, 6)
    ring.watch.drain()
    assert not ring.watch.pending and not ring.queue


def test_polling_waits_for_nothing(ring):
    for _ in range(3):
        ring.watch.after((b.OP_FWD,))
    ring.land(2)
    ring.watch.poll()
    assert len(ring.watch.pending) == 1


def test_an_error_is_raised_once_and_its_ring_is_empty_then(ring):
    for _ in range(4):
        ring.watch.after((b.OP_FWD,))
    ring.land()
    ring.land(code=b.ERR_RANGE)
    later(ring.land, 2, b.ERR_DEVICE_BOUNDS)
    with pytest.raises(b.Spa2Error) as e:
        ring.watch.poll()
    assert e.value.code == b.ERR_RANGE and not ring.watch.pending and not ring.queue
    ring.watch.drain()
    ring.watch.after((b.OP_FWD,))
    ring.land()
    ring.watch.poll()
    assert not ring.watch.pending
