"""RMS norm of every query and key row and the position rotation, in one pass:
what goes directly before the attention.

For a row x of d values: n = x / sqrt(mean(x^2) + eps), u = n * weight, and for
each pair (a, b) of the first ``rot_dim`` values, at the angle of its position,
(u_a cos - u_b sin, u_b cos + u_a sin).  ``forward`` and ``backward`` take
caller-owned outputs and workspace; ``norm_rotate`` is differentiable.  The
serving form, which writes keys and values into the pages of a cache, is
``paged.write``.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import layer
from .binding import lib


class RotaryParams(ctypes.Structure):
    """Mirror of ``elsaa_rotary_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "Hkv", "N", "d", "dtype", "rot_dim",
                                              "interleaved", "norm", "max_pos")] + \
               [("eps", ctypes.c_float)]

    @classmethod
    def make(cls, B, H, Hkv, N, d, dtype, rot_dim=None, max_pos=0, interleaved=False, norm=True,
             eps=1e-6) -> "RotaryParams":
        rot_dim = d if rot_dim is None else rot_dim
        return cls(B, H, Hkv, N, d, layer.dtype_code(dtype), rot_dim, int(bool(interleaved)),
                   int(bool(norm)), max_pos, float(eps))


def angle_table(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """(cos, sin) of position * base^(-2 i / rot_dim): fp32 [max_pos, rot_dim / 2, 2], from
    angles in 64 bits (a 32-bit angle of a far position has lost its fraction)."""
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack([ang.cos(), ang.sin()], dim=-1).to(torch.float32)


def validate(p: RotaryParams) -> int:
    return lib().elsaa_rotary_validate(ctypes.byref(p))


def workspace_bytes(p: RotaryParams) -> int:
    return lib().elsaa_rotary_workspace_bytes(ctypes.byref(p))


def alloc_workspace(p: RotaryParams, device) -> torch.Tensor:
    return layer.alloc_workspace(workspace_bytes(p), device)


def _shapes(p: RotaryParams):
    return (p.B, p.H, p.N, p.d), (p.B, p.Hkv, p.N, p.d)


def angles_and_weights(p: RotaryParams, table, q_weight, k_weight, dev):
    """The addresses of the checked table and weights, and what holds them."""
    if p.rot_dim == 0:
        table = None
    elif table is None:
        raise ValueError("rot_dim > 0 needs a table")
    at, _, held = layer.place(
        dev, 0, ("table", table, (p.max_pos, p.rot_dim // 2, 2), torch.float32, layer.as_small),
        ("q_weight", q_weight, (p.d,), torch.float32, layer.as_small),
        ("k_weight", k_weight, (p.d,), torch.float32, layer.as_small))
    return at, held


@layer.on_device(1)
def forward(p: RotaryParams, q, k, table=None, q_weight=None, k_weight=None, positions=None,
            qo=None, ko=None, ws=None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(qo, ko): q [B, H, N, d] and k [B, Hkv, N, d] (or None) normed and rotated.  Views with
    other strides (heads of a fused projection) are read in place."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    sq, sk = _shapes(p)
    if qo is None:
        qo = layer.like(q)
    if k is None:
        if ko is not None:
            raise ValueError("ko without k")
    elif ko is None:
        ko = layer.like(k)
    (pq, pk, pqo, pko), strides, _held = layer.place(
        dev, 3, ("q", q, sq, dt, layer.as_input), ("k", k, sk, dt, layer.as_input),
        ("qo", qo, sq, dt, layer.as_output), ("ko", ko, sk, dt, layer.as_output))
    (ptable, pwq, pwk), _small = angles_and_weights(p, table, q_weight, k_weight, dev)
    (ppos,), _, _pos = layer.place(dev, 0, ("positions", positions, (p.B, p.N), torch.int32,
                                            layer.as_small))
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p), dev)
    layer.ok("elsaa_rotary_forward", lib().elsaa_rotary_forward(
        ctypes.byref(p), pq, pk, strides, ppos, ptable, pwq, pwk, pqo, pko, ws.data_ptr(),
        ws.numel(), stream))
    return qo, ko


@layer.on_device(1)
def backward(p: RotaryParams, q, k, table, q_weight, k_weight, dqo, dko, positions=None, dq=None,
             dk=None, dq_weight=None, dk_weight=None, ws=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of sum(qo * dqo) + sum(ko * dko); the weights' gradients
    are None without the norm, dk's and dk_weight's without k."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    sq, sk = _shapes(p)
    if dq is None:
        dq = layer.like(q)
    if k is None:
        if dko is not None or dk is not None or dk_weight is not None:
            raise ValueError("dko, dk or dk_weight without k")
    elif dk is None:
        dk = layer.like(k)
    if not p.norm:
        if dq_weight is not None or dk_weight is not None:
            raise ValueError("gradients of weights without the norm")
    else:
        if dq_weight is None:
            dq_weight = torch.empty(p.d, dtype=torch.float32, device=dev)
        if k is not None and dk_weight is None:
            dk_weight = torch.empty(p.d, dtype=torch.float32, device=dev)
    into, out = layer.as_input, layer.as_output
    (pq, pk, pdqo, pdko, pdq, pdk), strides, _held = layer.place(
        dev, 3, ("q", q, sq, dt, into), ("k", k, sk, dt, into), ("dqo", dqo, sq, dt, into),
        ("dko", dko, sk, dt, into), ("dq", dq, sq, dt, out), ("dk", dk, sk, dt, out))
    (ptable, pwq, pwk), _small = angles_and_weights(p, table, q_weight, k_weight, dev)
    (ppos, pdwq, pdwk), _, _pos = layer.place(
        dev, 0, ("positions", positions, (p.B, p.N), torch.int32, layer.as_small),
        ("dq_weight", dq_weight, (p.d,), torch.float32, out),
        ("dk_weight", dk_weight, (p.d,), torch.float32, out))
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p), dev)
    layer.ok("elsaa_rotary_backward", lib().elsaa_rotary_backward(
        ctypes.byref(p), pq, pk, strides, ppos, ptable, pwq, pwk, pdqo, pdko, pdq, pdk, pdwq, pdwk,
        ws.data_ptr(), ws.numel(), stream))
    return dq, dk, dq_weight, dk_weight


class NormRotateFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run in libelsaa."""

    @staticmethod
    def forward(ctx, q, k, table, q_weight, k_weight, positions, params: RotaryParams, ws=None):
        qo, ko = forward(params, q, k, table, q_weight, k_weight, positions, ws=ws)
        ctx.params, ctx.ws = params, ws
        ctx.save_for_backward(q, k, table, q_weight, k_weight, positions)
        return qo, ko

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dqo, dko):
        q, k, table, q_weight, k_weight, positions = ctx.saved_tensors
        dq, dk, dwq, dwk = backward(ctx.params, q, k, table, q_weight, k_weight, dqo, dko,
                                    positions, ws=ctx.ws)
        return (dq, dk, None, dwq if q_weight is not None else None,
                dwk if k_weight is not None else None, None, None, None)


def norm_rotate(q, k, table=None, q_weight=None, k_weight=None, positions=None, rot_dim=None,
                interleaved=False, norm=True, eps=1e-6, ws=None):
    """Differentiable norm and rotation of q [B, H, N, d] and k [B, Hkv, N, d]; ``table`` as
    ``angle_table`` makes it (None: norm only), with a row for every token where there are no int32
    ``positions`` [B, N].  The weights are fp32 [d] (None: ones) and belong to the norm: without it
    they are not used.  ``ws`` (``alloc_workspace``) serves the forward and the backward; what they
    record on the device (positions outside the table, whose rows are zeros) is read with
    ``binding.check(ws)``.  Without it each makes its own, and the record is lost with it.  In a
    captured step as ``window.window_attention``."""
    B, H, N, d = q.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, Hkv, N, d]")
    if rot_dim is None:
        rot_dim = 0 if table is None else 2 * table.shape[1]
    p = RotaryParams.make(B, H, k.shape[1], N, d, q.dtype, rot_dim,
                          0 if table is None else table.shape[0], interleaved, norm, eps)
    return NormRotateFunction.apply(q, k, table, q_weight, k_weight, positions, p, ws)


class QkRotary(NamedTuple):
    """How ``binding.elsaa`` norms and rotates q and k before the operator (its ``rotary``)."""
    table: Optional[torch.Tensor] = None
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    positions: Optional[torch.Tensor] = None
    interleaved: bool = False
    norm: bool = True
    eps: float = 1e-6
    ws: Optional[torch.Tensor] = None

    def apply(self, q, k):
        return norm_rotate(q, k, self.table, self.q_weight, self.k_weight, self.positions,
                           interleaved=self.interleaved, norm=self.norm, eps=self.eps, ws=self.ws)
