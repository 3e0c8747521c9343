"""What rotary.py, window.py and paged.py share: argument checks, strides and
the call into libelsaa on the tensors' own device."""

from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from . import binding
from .binding import ELSAA_BF16, ELSAA_F32

_TORCH = {ELSAA_BF16: torch.bfloat16, ELSAA_F32: torch.float32}


def dtype_code(dtype) -> int:
    """elsaa_dtype of "bf16" / "f32" or the torch dtype."""
    if dtype in ("bf16", torch.bfloat16):
        return ELSAA_BF16
    if dtype in ("f32", torch.float32):
        return ELSAA_F32
    raise TypeError(f"dtype must be bf16 or f32, got {dtype}")


def torch_dtype(code: int) -> torch.dtype:
    return _TORCH[code]


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace with its head cleared (the error word and the counters)."""
    if nbytes == 0:
        raise ValueError("not a valid problem")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:8192].zero_()
    return ws


def check(where: str, t: torch.Tensor, shape: Sequence[int], dtype: torch.dtype,
          device: torch.device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{where}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{where}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{where}: on {t.device}, expected {device}")


def strided(t: torch.Tensor) -> bool:
    """Whether the library takes the tensor where it lies: the last dimension
    contiguous, the other strides multiples of 16 bytes and at least a row, the
    start on 16 bytes."""
    if t.data_ptr() & 15:
        return False
    if t.is_contiguous():
        return True
    e, d = t.element_size(), t.shape[-1]
    return t.stride(-1) == 1 and all(n == 1 or (s >= d and s * e % 16 == 0)
                                     for n, s in zip(t.shape[:-1], t.stride()[:-1]))


def rows_apart(t: torch.Tensor) -> bool:
    """Whether no two elements of a strided tensor share memory (by its dimensions one inside
    the other, as every view of a dense tensor has them)."""
    if t.is_contiguous():
        return True
    end = 0                # the last offset of the smaller strides' dimensions
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if s <= end:
            return False
        end += s * (n - 1)
    return True


def like(t: torch.Tensor) -> torch.Tensor:
    """A new dense tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def as_input(where: str, t: torch.Tensor, shape, dtype, device) -> torch.Tensor:
    """The checked tensor, or a dense copy of one the library does not take
    where it lies (a broadcast one, an odd stride or offset)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        check(where, t, shape, dtype, device)
    if t.is_contiguous() and not t.data_ptr() & 15 or strided(t):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def as_output(where: str, t: torch.Tensor, shape, dtype, device) -> torch.Tensor:
    """The checked output, refused where the library does not take it where it lies."""
    check(where, t, shape, dtype, device)
    if not strided(t) or not rows_apart(t):
        raise ValueError(f"{where}: an output needs a contiguous last dimension, strides and a "
                         "start that are multiples of 16 bytes, and no two elements in one place")
    return t


def as_small(where: str, t: torch.Tensor, shape, dtype, device) -> torch.Tensor:
    """The checked int32 / fp32 tensor, dense and on 16 bytes (copied where it is not)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        check(where, t, shape, dtype, device)
    if t.is_contiguous() and not t.data_ptr() & 15:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def as_workspace(ws: Optional[torch.Tensor], nbytes, device) -> torch.Tensor:
    """The caller's workspace (the library checks its size), or a new one of nbytes()."""
    if ws is None:
        return alloc_workspace(nbytes(), device)
    if ws.device != device:
        raise ValueError(f"ws: on {ws.device}, expected {device}")
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous uint8 tensor")
    return ws


def place(device: torch.device, dims: int, *specs):
    """The addresses of a call's tensors, the strides of their first ``dims`` dimensions (None:
    all are dense) and what has to live until the launch.  A spec is (name, tensor or None, shape,
    dtype, how): ``how`` (as_input, as_output, ...) checks and places a tensor that is not dense
    and on 16 bytes.  (One pass over the tensors: a call's host time is mostly these checks.)"""
    at = []
    for _, t, shape, dtype, _ in specs:
        if t is None:
            at.append(None)
        elif t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
            p = t.data_ptr()
            if p & 15:
                break
            at.append(p)
        else:
            break
    else:
        return at, None, None
    held = [t if t is None else how(where, t, shape, dtype, device)
            for where, t, shape, dtype, how in specs]
    return [None if t is None else t.data_ptr() for t in held], strides_of(dims, *held), held


def strides_of(dims: int, *tensors: Optional[torch.Tensor]):
    """Host array of the first `dims` strides of every tensor, or None where
    all are dense."""
    for t in tensors:
        if t is not None and not t.is_contiguous():
            break
    else:
        return None
    flat = []
    for t in tensors:
        flat += [0] * dims if t is None else t.stride()[:dims]
    return (ctypes.c_int64 * len(flat))(*flat)


# the current stream's handle without a Stream object around it
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


def on_device(at: int):
    """Decorator of the entry points f(..., q, ..., stream=None), q the argument number ``at``:
    runs f with q's device current and the given stream (or the device's current one) current
    for its allocations; f gets the raw stream."""
    def wrap(f):
        @functools.wraps(f)
        def call(*args, stream=None, **kw):
            device = (args[at] if len(args) > at else kw["q"]).device
            if device.type != "cuda":
                raise ValueError(f"tensors must be on a CUDA device, got {device}")
            if stream is None:
                if device.index == torch.cuda.current_device():
                    return f(*args, stream=_raw_stream(device.index), **kw)
                with torch.cuda.device(device):
                    return f(*args, stream=_raw_stream(device.index), **kw)
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            with torch.cuda.device(device), torch.cuda.stream(stream):
                return f(*args, stream=stream.cuda_stream, **kw)

        return call

    return wrap


def ok(where: str, code: int) -> None:
    if code != 0:
        raise binding.ElsaaError(where, code)
