"""Activation checkpoints in 8 bits.

    kept = pack8(q, k, v)        # one launch; 33/32 bytes per element
    q2, k2, v2 = unpack8(*kept)  # the kept values, in the tensors' own type

Every group of 32 consecutive elements of a row (of the last dimension; the last
group of a row may be shorter) is held as one int8 code per element and one
exponent byte, the exponent of the group's largest magnitude. A code counts
power-of-two steps of 1/64 to 1/128 of that magnitude, so a kept value is off by at
most half a step (less than one at the very top of a group, where codes are clamped
to 127), and reading it back is exact in bf16, fp16 and fp32. A group that held an
infinity or a NaN reads back as NaN.

`sparse_attention(..., checkpoint="int8")` keeps its q, k, v this way for the backward
pass. `pack8` and `unpack8` are for whatever else a training step holds between
its passes; they are not differentiable (they return detached tensors) and may be
captured into a CUDA graph.
"""

from __future__ import annotations

import torch

from . import binding as b

_DTYPES = {torch.bfloat16: b.DTYPE_BF16, torch.float32: b.DTYPE_F32, torch.float16: b.DTYPE_F16}


class Packed:
    """One tensor as 8-bit codes and exponent bytes, both in one device buffer."""

    __slots__ = ("data", "shape", "dtype")

    def __init__(self, data: torch.Tensor, shape, dtype: torch.dtype):
        self.data, self.shape, self.dtype = data, torch.Size(shape), dtype

    @staticmethod
    def _sizes(shape):
        d = shape[-1]
        n = shape.numel()
        return n, -(-n // 16) * 16, (n // d) * -(-d // b.PACK8_GROUP) if n else 0

    @classmethod
    def empty_like(cls, x: torch.Tensor) -> "Packed":
        _, at, groups = cls._sizes(x.shape)
        return cls(torch.empty(at + groups, dtype=torch.uint8, device=x.device), x.shape, x.dtype)

    @property
    def codes(self) -> torch.Tensor:
        """int8 codes, in the tensor's shape."""
        return self.data[:self._sizes(self.shape)[0]].view(torch.int8).view(self.shape)

    @property
    def exponents(self) -> torch.Tensor:
        """uint8 biased exponents [..., ceil(d / 32)]."""
        _, at, groups = self._sizes(self.shape)
        return self.data[at:at + groups].view(*self.shape[:-1], -(-self.shape[-1] // b.PACK8_GROUP))

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    def c(self, x: torch.Tensor | None = None) -> b.spa2_pack8_tensor:
        n, at, _ = self._sizes(self.shape)
        p, d = self.data.data_ptr(), self.shape[-1]
        return b.spa2_pack8_tensor(None if x is None else x.data_ptr(), p, p + at, n // d, d)


def _launch(call, items, dtype, device, what):
    """`items`: (Packed, tensor) pairs, at most PACK8_MAX to a launch, on the device's current stream."""
    with b.on_device(device):
        s = torch.cuda.current_stream().cuda_stream
        for i in range(0, len(items), b.PACK8_MAX):
            part = items[i:i + b.PACK8_MAX]
            b._check(call((b.spa2_pack8_tensor * len(part))(*(p.c(x) for p, x in part)), _DTYPES[dtype], s), what)


def _same(items, what):
    if not items:
        raise ValueError(f"{what} expects at least one tensor")
    first = items[0]
    if any(x.dtype != first.dtype for x in items):
        raise TypeError(f"{what} expects tensors of one dtype")


def pack8(*xs: torch.Tensor) -> tuple[Packed, ...]:
    """8-bit checkpoints of CUDA tensors of one dtype (bf16, fp16 or fp32) and any shapes."""
    _same(xs, "pack8")
    if xs[0].dtype not in _DTYPES:
        raise TypeError(f"pack8 expects bf16, fp16 or fp32 tensors, got {xs[0].dtype}")
    if any(x.device != xs[0].device or x.device.type != "cuda" for x in xs):
        raise ValueError("pack8 expects tensors on one CUDA device")
    if any(x.dim() < 1 or x.shape[-1] < 1 for x in xs):
        raise ValueError("pack8 expects tensors of at least one dimension, the last of them not empty")
    items = [(Packed.empty_like(x), x.detach().contiguous()) for x in xs]
    _launch(b.spa2_pack8, items, xs[0].dtype, xs[0].device, "spa2_pack8")
    return tuple(p for p, _ in items)


def unpack8(*packed: Packed) -> tuple[torch.Tensor, ...]:
    """The kept values of each checkpoint, contiguous, in its tensor's shape and dtype."""
    _same(packed, "unpack8")
    device = packed[0].data.device
    if any(p.data.device != device for p in packed):
        raise ValueError("unpack8 expects checkpoints on one CUDA device")
    items = [(p, torch.empty(p.shape, dtype=p.dtype, device=device)) for p in packed]
    _launch(b.spa2_unpack8, items, packed[0].dtype, device, "spa2_unpack8")
    return tuple(x for _, x in items)
