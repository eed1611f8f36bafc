"""`torch.autograd` front end of the sparse attention path.

sparse_attention(q, k, v, k_frac, p_frac) builds the hybrid Top-k + Top-p block
mask of (q, k) (paper.rainbus.top summary, 方法步骤详情 steps 1-3), runs the
block-sparse forward (step 4) and, when a gradient is requested, the backward
through the same mask, which the method holds constant (its trainable part is
the attention itself: chatpaper.ai abstract (ii)). Every step runs in the
libspa2 kernels; this module only marshals arguments through the C ABI
(`binding.Spa2`) and caches the per-shape workspaces.

A mask can also be built once with `block_mask(q, k, k_frac, p_frac)` and
passed as `sparse_attention(..., mask=m)` to later calls of the same shape
(other diffusion steps or layers), which then skip pooling and selection.

Device-side errors (a bounds check that failed on a bad mask, V outside the
fp16 range, a wait that timed out) are reported without synchronising the
stream: after every call the status words are copied, in stream order, into
pinned host memory; the next call on that shape and stream raises `Spa2Error`
once such a copy has landed with an error in it, and `check_errors()` waits for
every pending copy and raises.

Workspaces are cached per (shape, device, CUDA stream) and allocated when an operation
first needs one: calls on different streams never share scratch memory. Host threads
that share a stream share its workspaces; a lock keeps the launches of one operation
together. A call that is captured into a CUDA graph gets workspaces of its own, from the
graph's memory, and its device-side errors are not reported (a replay reads no status
word). As for any torch operator, a captured backward pass wants leaves that no live
eager graph holds (torch ends the capture with an exception otherwise).

`sparse_attention(..., checkpoint="int8")` keeps q, k and v for the backward pass as
8-bit checkpoints (module `checkpoint`) and the mask's lists, nothing else of their
size; the backward pass computes the attention again from the kept values and returns
its gradients there. `rotary=` turns q and k by their positions first (module `rotary`).
"""

from __future__ import annotations

import threading
import time
from collections import deque

import torch

from . import binding as b
from .checkpoint import Packed, _check_not_traced
from .rotary import Rotary, apply_rotary

_cache: dict = {}
_cache_lock = threading.Lock()


class _StatusWatch:
    """Stream-ordered, non-blocking copies of one Spa2's status words into pinned memory. A
    slot holds PENDING until its copy lands, so a look at it needs no event. Used under the
    Spa2's lock."""

    SLOTS, PENDING = 16, -1

    def __init__(self, spa: b.Spa2):
        self.spa = spa
        self.host = torch.zeros(self.SLOTS, 3, dtype=torch.int32).pin_memory()
        self.codes = self.host.numpy()
        self.pending: deque = deque()      # (slot, ops) in launch order
        self.next = 0

    def after(self, ops):
        """Queue a copy of the status words of `ops` behind the work just launched."""
        if len(self.pending) == self.SLOTS:
            self._finish()
        slot = self.next
        self.next = (self.next + 1) % self.SLOTS
        at, stream = self.host.data_ptr() + 12 * slot, b._stream(torch)
        for col, op in enumerate(ops):
            self.codes[slot, col] = self.PENDING
            b._check(b.spa2_status_fetch(self.spa.ws[op].data_ptr(), at + 4 * col, stream), "spa2_status_fetch")
        self.pending.append((slot, ops))

    def poll(self):
        """Raise the first error among copies that have landed (never waits for one that has not, but once
        there is an error, for the others of this stream)."""
        while self.pending and self._landed():
            self._finish()

    def drain(self):
        """Wait for every pending copy, then raise the first error among them."""
        while self.pending:
            self._finish()

    def _landed(self):
        slot, ops = self.pending[0]
        return self.codes[slot, len(ops) - 1] != self.PENDING   # the copies of a slot land in order

    def _wait(self):
        """Until the oldest pending copy has landed: by looking at its word, so that nothing but the work in front
        of it is waited for, on this stream or another (an event for every call would cost each of them a
        microsecond). A copy that a failed context will never make ends the wait with that failure."""
        pause, check_at = 2e-5, time.monotonic() + 0.5
        while not self._landed():
            time.sleep(pause)
            pause = min(2 * pause, 2e-4)
            if time.monotonic() > check_at:
                check_at += 0.5
                if not torch.cuda.is_current_stream_capturing():   # a query would end the capture
                    torch.cuda.current_stream(self.spa.device).query()

    def _finish(self):
        if not self._landed():
            self._wait()
        slot, ops = self.pending.popleft()
        for col, op in enumerate(ops):
            code = int(self.codes[slot, col])
            if code != b.OK:
                while self.pending:   # this stream's other calls: only the first error is raised
                    self._wait()
                    self.pending.popleft()
                raise b.Spa2Error(code, f"device status of sparse_attention (op {op})")


class _NoWatch:
    """In the place of a _StatusWatch while a CUDA graph is captured: neither event
    queries nor copies that a replay would repeat into a stale slot."""

    def after(self, ops):
        pass

    def poll(self):
        pass


def _spa(B, H, N, d, device, bq=b.BQ, bkv=b.BKV) -> b.Spa2:
    """The Spa2 of this shape and the current stream. An operation on it holds its `lock` from the first launch to
    the status copy: the kernels of one C call hand each other data through the workspace, and another thread's
    launches on the same stream must not come between them."""
    if torch.cuda.is_current_stream_capturing():
        # graphs replay on any stream, two of them at once: each call owns its workspaces
        s = b.Spa2(B, H, N, d, device=device, bq=bq, bkv=bkv, lazy=True)
        s.watch = _NoWatch()
        return s
    index = torch.cuda.current_device() if device.index is None else device.index
    key = (B, H, N, d, bq, bkv, index, torch._C._cuda_getCurrentRawStream(index))
    s = _cache.get(key)
    if s is None:
        with _cache_lock:
            s = _cache.get(key)
            if s is None:
                s = b.Spa2(B, H, N, d, device=device, bq=bq, bkv=bkv, lazy=True)
                s.watch = _StatusWatch(s)
                _cache[key] = s
    return s


def check_errors():
    """Wait for every pending status copy of every cached workspace and raise
    `Spa2Error` if any call of sparse_attention / block_mask recorded a
    device-side error."""
    for s in list(_cache.values()):
        with s.lock:
            s.watch.drain()


class SparseAttentionFunction(torch.autograd.Function):
    """O = block-sparse attention of (q, k, v) under the hybrid mask of (q, k).

    q, k, v: [B, H, N, d] bf16 CUDA tensors (d in {64, 128}); gradients come back
    in bf16. The mask of the last call is kept on the function's context (and
    returned by `sparse_attention(..., return_mask=True)`).
    """

    @staticmethod
    def forward(ctx, q, k, v, k_frac: float, p_frac: float, scale: float = 0.0, mask: b.Mask | None = None,
                bq: int = b.BQ, bkv: int = b.BKV):
        if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
            raise TypeError("sparse_attention expects bf16 q, k, v")
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        B, H, N, d = q.shape
        s = _spa(B, H, N, d, q.device, bq, bkv)
        ops = [b.OP_FWD]
        if mask is not None and (tuple(mask.row_cnt.shape) != (B, H, s.Tm) or tuple(mask.row_idx.shape) != (B, H, s.Tm, s.Tn)
                                 or mask.col_cnt is None or mask.row_cnt.device != q.device):
            raise ValueError("mask does not belong to a problem of this shape and device")
        with s.lock:
            s.watch.poll()
            if mask is None:
                mask = s.block_mask(q, k, k_frac, p_frac)
                ops.insert(0, b.OP_MASK)
            o, lse = s.fwd(q, k, v, mask, scale)
            o_lo = s.o_lo
            s.watch.after(ops)
        ctx.save_for_backward(q, k, v, o, lse, o_lo)
        ctx.mask, ctx.scale, ctx.spa = mask, scale, s
        row_cnt = mask.row_cnt.clone()  # the kept-block counts (a copy: a reused mask serves many calls)
        ctx.mark_non_differentiable(row_cnt)
        return o, row_cnt

    @staticmethod
    def backward(ctx, do, _row_cnt_grad):
        q, k, v, o, lse, o_lo = ctx.saved_tensors
        spa = ctx.spa
        if torch.cuda.is_current_stream_capturing():
            spa = _spa(spa.B, spa.H, spa.N, spa.d, spa.device, spa.bq, spa.bkv)
        do = do.contiguous()
        with spa.lock:
            spa.watch.poll()
            dq, dk, dv = spa.bwd(q, k, v, o, lse, do, ctx.mask, ctx.scale, o_lo=o_lo, grad_dtype=b.DTYPE_BF16)
            spa.watch.after([b.OP_BWD])
        return dq, dk, dv, None, None, None, None, None, None


class CheckpointedAttentionFunction(torch.autograd.Function):
    """SparseAttentionFunction with q, k, v kept in 8 bits for the backward pass: the
    same o, and the gradients of the attention at the kept values."""

    @staticmethod
    def forward(ctx, q, k, v, scale: float, mask: b.Mask, bq: int, bkv: int):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        s = _spa(*q.shape, q.device, bq, bkv)
        with s.lock:
            s.watch.poll()
            o, kept = s.fwd_ckpt(q, k, v, mask, scale)
            s.watch.after((b.OP_FWD,))
        ctx.save_for_backward(kept[0].base)
        ctx.mask, ctx.scale, ctx.spa = mask.lists(), scale, s
        ctx.versions = ctx.mask.versions()
        return o

    @staticmethod
    def backward(ctx, do):
        if torch.is_grad_enabled():  # wanted as a part of a graph, which cannot be differentiated again
            return _checkpointed_backward_in_graph(ctx, do)
        return _checkpointed_backward(ctx, do)


def _checkpointed_backward(ctx, do):
    s = ctx.spa
    if ctx.mask.versions() != ctx.versions:
        raise RuntimeError("the lists of the block mask were changed in place after sparse_attention: the backward pass "
                           "would be that of another attention than the one whose o it returned")
    if torch.cuda.is_current_stream_capturing():
        s = _spa(s.B, s.H, s.N, s.d, s.device, s.bq, s.bkv)
    kept, do = Packed.several_in(ctx.saved_tensors[0], do.shape, do.dtype, 3), do.contiguous()
    with s.lock:
        s.watch.poll()
        grads = s.bwd_ckpt(kept, do, ctx.mask, ctx.scale, grad_dtype=b.DTYPE_BF16)
        s.watch.after((b.OP_BWD_CKPT,))
    return (*grads, None, None, None, None)


_checkpointed_backward_in_graph = torch.autograd.function.once_differentiable(_checkpointed_backward)


def _check_attention(q, k, v, mask, bq, bkv):
    """What the checkpointed call checks before it touches the device."""
    if not q.dtype == k.dtype == v.dtype == torch.bfloat16:
        raise TypeError("sparse_attention expects bf16 q, k, v")
    shape, device = q.shape, q.device
    if len(shape) != 4 or k.shape != shape or v.shape != shape:
        raise ValueError("sparse_attention expects q, k, v of one shape [B, H, N, d]")
    if device.type != "cuda" or k.device != device or v.device != device:
        raise ValueError("sparse_attention expects q, k, v on one CUDA device")
    if mask is not None:
        B, H, N, _ = shape
        Tm, Tn = b.block_counts(N, bq, bkv)
        for t, want in ((mask.row_cnt, (B, H, Tm)), (mask.row_idx, (B, H, Tm, Tn)), (mask.col_cnt, (B, H, Tn)),
                        (mask.col_idx, (B, H, Tn, Tm))):
            if t is None or t.shape != want or t.device != device or t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("mask must be int32 lists, contiguous, of a problem of this shape and device")


def block_mask(q, k, k_frac: float, p_frac: float, bq: int = b.BQ, bkv: int = b.BKV) -> b.Mask:
    """The hybrid block mask of (q, k) alone (CSR and CSC on the device), for
    reuse through `sparse_attention(..., mask=...)`."""
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16:
        raise TypeError("block_mask expects bf16 q, k")
    q, k = q.contiguous(), k.contiguous()
    B, H, N, d = q.shape
    with b.on_device(q.device):
        s = _spa(B, H, N, d, q.device, bq, bkv)
        with s.lock:
            s.watch.poll()
            m = s.block_mask(q, k, k_frac, p_frac)
            s.watch.after([b.OP_MASK])
    return m


def sparse_attention(q, k, v, k_frac: float = 0.0, p_frac: float = 0.0, scale: float = 0.0,
                     return_mask: bool = False, mask: b.Mask | None = None, bq: int = b.BQ, bkv: int = b.BKV,
                     checkpoint: str | None = None, rotary: Rotary | None = None):
    """Differentiable hybrid block-sparse attention with query blocks of bq rows
    (64, 128 or 256) and key/value blocks of bkv rows (64 or 128).

    With `mask` (from `block_mask` on a problem of the same shape and block
    sizes) the given mask is used as is and k_frac, p_frac are ignored.

    checkpoint="int8" keeps q, k, v in 8 bits for the backward pass (3.1 bytes per
    element of q in place of 10) and computes the attention again there: the same o,
    and its gradients at the kept values. Where no gradient is wanted nothing is kept.
    The mask's lists must not change before the backward pass, which raises if they did.

    `rotary` turns q and k before the mask and the attention; the mask given by
    `mask` is one of turned q and k.
    """
    if checkpoint not in (None, "int8"):
        raise ValueError(f"unknown checkpoint {checkpoint!r}: None or 'int8'")
    if checkpoint is not None:
        _check_not_traced("sparse_attention with a checkpoint")
    if rotary is not None:
        q, k = apply_rotary(q, k, inv_freq=rotary.inv_freq, positions=rotary.positions, layout=rotary.layout,
                            axes=rotary.axes, scale=rotary.scale)
    with b.on_device(q.device):
        if checkpoint is not None:
            _check_attention(q, k, v, mask, bq, bkv)
            if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
                if mask is None:
                    q, k = q.contiguous(), k.contiguous()  # once for both
                    mask = block_mask(q, k, k_frac, p_frac, bq, bkv)
                o = CheckpointedAttentionFunction.apply(q, k, v, scale, mask, bq, bkv)
                return (o, mask.row_cnt.clone()) if return_mask else o
        o, row_cnt = SparseAttentionFunction.apply(q, k, v, k_frac, p_frac, scale, mask, bq, bkv)
    return (o, row_cnt) if return_mask else o
