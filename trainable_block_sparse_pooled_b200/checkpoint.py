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
its passes; they are not differentiable (they return detached tensors; inputs with a
forward-mode tangent are refused, and so are traces of torch.jit) and may be captured
into a CUDA graph.
"""

from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import binding as b

_DTYPES = {torch.bfloat16: b.DTYPE_BF16, torch.float32: b.DTYPE_F32, torch.float16: b.DTYPE_F16}


class Packed:
    """One tensor as 8-bit codes and exponent bytes, both in one device buffer (or a part of it)."""

    __slots__ = ("base", "offset", "shape", "dtype")

    def __init__(self, base: torch.Tensor, shape, dtype: torch.dtype, offset: int = 0):
        self.base, self.offset, self.shape, self.dtype = base, offset, shape, dtype

    @staticmethod
    def _sizes(shape):
        """(elements, byte at which the exponents begin, exponents)"""
        d, n = shape[-1], shape.numel()
        return n, (n + 15) & ~15, n // d * ((d + 31) >> 5)

    @classmethod
    def empty_like(cls, x: torch.Tensor) -> "Packed":
        shape = x.shape
        _, at, groups = cls._sizes(shape)
        return cls(x.new_empty(at + groups, dtype=torch.uint8), shape, x.dtype)

    @classmethod
    def several_like(cls, x: torch.Tensor, n: int) -> tuple:
        """n checkpoints of tensors like x in one buffer."""
        _, at, groups = cls._sizes(x.shape)
        size = n * ((at + groups + 15) & ~15)
        return cls.several_in(x.new_empty(size, dtype=torch.uint8), x.shape, x.dtype, n)

    @classmethod
    def several_in(cls, base, shape, dtype, n) -> tuple:
        return tuple([cls(base, shape, dtype, i * (base.shape[0] // n)) for i in range(n)])

    @property
    def data(self) -> torch.Tensor:
        """The bytes: codes, padded to a multiple of 16, then exponents."""
        return self.base[self.offset:self.offset + self.nbytes]

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
        _, at, groups = self._sizes(self.shape)
        return at + groups

    def fields(self, x: torch.Tensor | None = None) -> tuple:
        """The fields of a spa2_pack8_tensor of this checkpoint and x (contiguous, of its shape)."""
        n, at, _ = self._sizes(self.shape)
        p, d = self.base.data_ptr() + self.offset, self.shape[-1]
        return 0 if x is None else x.data_ptr(), p, p + at, n // d, d

    def c(self, x: torch.Tensor | None = None) -> b.spa2_pack8_tensor:
        return b.spa2_pack8_tensor(*self.fields(x))


def _launch(call, items, dtype, device, what):
    """`items`: (Packed, tensor) pairs, at most PACK8_MAX to a launch, on the device's current stream."""
    for i in range(0, len(items), b.PACK8_MAX):
        part = items[i:i + b.PACK8_MAX]
        fields = []
        for p, x in part:
            fields += p.fields(x)
        rc = b.launch(call, device, b.PACK8_TENSORS[len(part)].pack(*fields), len(part), _DTYPES[dtype])
        if rc != b.OK:
            raise b.Spa2Error(rc, what)


def _check_not_traced(what):
    if torch.jit.is_tracing():
        raise RuntimeError(f"{what} cannot be traced: a trace would hold its buffers and not what fills them")


def pack8(*xs: torch.Tensor) -> tuple[Packed, ...]:
    """8-bit checkpoints of CUDA tensors of one dtype (bf16, fp16 or fp32) and any shapes."""
    if not xs:
        raise ValueError("pack8 expects at least one tensor")
    _check_not_traced("pack8")
    dtype, device = xs[0].dtype, xs[0].device
    if dtype not in _DTYPES:
        raise TypeError(f"pack8 expects bf16, fp16 or fp32 tensors, got {dtype}")
    for x in xs:
        if x.dtype != dtype:
            raise TypeError("pack8 expects tensors of one dtype")
    items = []
    for x in xs:
        if x.device != device or device.type != "cuda":
            raise ValueError("pack8 expects tensors on one CUDA device")
        if x.dim() < 1 or x.shape[-1] < 1:
            raise ValueError("pack8 expects tensors of at least one dimension, the last of them not empty")
        if forward_ad._current_level >= 0 and forward_ad.unpack_dual(x).tangent is not None:
            raise RuntimeError("pack8 has no forward-mode derivative")
        items.append((Packed.empty_like(x), x if x.is_contiguous() else x.detach().contiguous()))
    _launch(b.lib().spa2_pack8, items, dtype, device, "spa2_pack8")
    return tuple([p for p, _ in items])


def unpack8(*packed: Packed) -> tuple[torch.Tensor, ...]:
    """The kept values of each checkpoint, contiguous, in its tensor's shape and dtype."""
    if not packed:
        raise ValueError("unpack8 expects at least one checkpoint")
    _check_not_traced("unpack8")
    dtype, device = packed[0].dtype, packed[0].base.device
    for p in packed:
        if p.dtype != dtype:
            raise TypeError("unpack8 expects checkpoints of tensors of one dtype")
    for p in packed:
        if p.base.device != device or device.type != "cuda":
            raise ValueError("unpack8 expects checkpoints on one CUDA device")
        if p.base.dtype != torch.uint8 or not p.base.is_contiguous() or p.base.numel() - p.offset < p.nbytes:
            raise ValueError("unpack8 expects checkpoints as pack8 makes them")
    items = [(p, p.base.new_empty(p.shape, dtype=dtype)) for p in packed]
    _launch(b.lib().spa2_unpack8, items, dtype, device, "spa2_unpack8")
    return tuple([x for _, x in items])
