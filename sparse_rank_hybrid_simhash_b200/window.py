"""Exact causal attention over a sliding window of tokens with sinks, forward and
backward.

Query i sees the keys j <= i with i - j < window (0: all of them) or j < sinks.
Hkv key heads serve H query heads (query head h reads key head h // (H // Hkv)).
A padded batch gives its ``lengths``: rows at or behind a length take part in
nothing, their output and gradients are zero and their lse is -inf.  ``forward``
and ``backward`` take caller-owned outputs and workspace; ``window_attention`` is
differentiable.  The serving form over a paged cache is ``paged.attend``.
"""

from __future__ import annotations

import ctypes
from typing import Tuple

import torch

from . import layer
from .binding import lib


class WindowParams(ctypes.Structure):
    """Mirror of ``elsaa_window_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "Hkv", "N", "d", "dtype", "window",
                                              "sinks")] + [("scale", ctypes.c_float)]

    @classmethod
    def make(cls, B, H, Hkv, N, d, dtype, window=0, sinks=0, scale=0.0) -> "WindowParams":
        return cls(B, H, Hkv, N, d, layer.dtype_code(dtype), window, sinks, float(scale))


def validate(p: WindowParams) -> int:
    return lib().elsaa_window_validate(ctypes.byref(p))


def workspace_bytes(p: WindowParams, backward: bool = True) -> int:
    return lib().elsaa_window_workspace_bytes(ctypes.byref(p), int(backward))


def alloc_workspace(p: WindowParams, device, backward: bool = True) -> torch.Tensor:
    return layer.alloc_workspace(workspace_bytes(p, backward), device)


def _shapes(p: WindowParams):
    return (p.B, p.H, p.N, p.d), (p.B, p.Hkv, p.N, p.d)


def _as_lse(where, t, shape, dtype, device):
    layer.check(where, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{where} must be contiguous")
    return t


@layer.on_device(1)
def forward(p: WindowParams, q, k, v, lengths=None, y=None, lse=None, ws=None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(y [B, H, N, d], lse [B, H, N] fp32).  Views of q, k, v, y with other strides are taken
    in place."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    sq, sk = _shapes(p)
    if y is None:
        y = layer.like(q)
    if lse is None:
        lse = torch.empty(sq[:3], dtype=torch.float32, device=dev)
    (pq, pk, pv, py), strides, _held = layer.place(
        dev, 3, ("q", q, sq, dt, layer.as_input), ("k", k, sk, dt, layer.as_input),
        ("v", v, sk, dt, layer.as_input), ("y", y, sq, dt, layer.as_output))
    (plse, plen), _, _small = layer.place(
        dev, 0, ("lse", lse, sq[:3], torch.float32, _as_lse),
        ("lengths", lengths, (p.B,), torch.int32, layer.as_small))
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p, False), dev)
    layer.ok("elsaa_window_forward", lib().elsaa_window_forward(
        ctypes.byref(p), pq, pk, pv, strides, plen, py, plse, ws.data_ptr(), ws.numel(), stream))
    return y, lse


@layer.on_device(1)
def backward(p: WindowParams, q, k, v, y, lse, dy, lengths=None, dq=None, dk=None, dv=None,
             ws=None, stream=None):
    """(dq, dk, dv) of sum(y * dy), from the y and lse of ``forward`` on the same inputs."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    sq, sk = _shapes(p)
    dq = layer.like(q) if dq is None else dq
    dk = layer.like(k) if dk is None else dk
    dv = layer.like(v) if dv is None else dv
    into, out = layer.as_input, layer.as_output
    (pq, pk, pv, py, pdy, pdq, pdk, pdv), strides, _held = layer.place(
        dev, 3, ("q", q, sq, dt, into), ("k", k, sk, dt, into), ("v", v, sk, dt, into),
        ("y", y, sq, dt, into), ("dy", dy, sq, dt, into), ("dq", dq, sq, dt, out),
        ("dk", dk, sk, dt, out), ("dv", dv, sk, dt, out))
    (plse, plen), _, _small = layer.place(
        dev, 0, ("lse", lse, sq[:3], torch.float32, layer.as_small),
        ("lengths", lengths, (p.B,), torch.int32, layer.as_small))
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p, True), dev)
    layer.ok("elsaa_window_backward", lib().elsaa_window_backward(
        ctypes.byref(p), pq, pk, pv, strides, plen, py, plse, pdy, pdq, pdk, pdv, ws.data_ptr(),
        ws.numel(), stream))
    return dq, dk, dv


class WindowFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run in libelsaa."""

    @staticmethod
    def forward(ctx, q, k, v, lengths, params: WindowParams, ws=None):
        y, lse = forward(params, q, k, v, lengths, ws=ws)
        ctx.params, ctx.ws = params, ws
        ctx.save_for_backward(q, k, v, y, lse, lengths)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        q, k, v, y, lse, lengths = ctx.saved_tensors
        return (*backward(ctx.params, q, k, v, y, lse, dy, lengths, ws=ctx.ws), None, None, None)


def window_attention(q, k, v, window=0, sinks=0, lengths=None, scale=0.0, ws=None):
    """Differentiable window attention of q [B, H, N, d] over k, v [B, Hkv, N, d]; ``lengths``
    int32 [B] on the device.

    ``ws`` (``alloc_workspace``) serves the forward and the backward; what they record on the
    device (a wait that gave up) is read with ``binding.check(ws)``.  Without it each makes its
    own, and the record is lost with it.

    A step captured in a CUDA graph must find no eager autograd graph of the same leaves alive
    (an output not yet dropped or detached): autograd would sum their gradients on that graph's
    stream, which breaks the capture."""
    B, H, N, d = q.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, Hkv, N, d]")
    p = WindowParams.make(B, H, k.shape[1], N, d, q.dtype, window, sinks, scale)
    return WindowFunction.apply(q, k, v, lengths, p, ws)
