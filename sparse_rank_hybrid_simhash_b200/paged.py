"""The serving forms over a cache in pages: ``write`` norms and rotates new tokens'
queries and keys and stores keys and values in the pages, ``attend`` is the
attention of those tokens (one or many a sequence) over the cache, with an
optional window and sinks.

The rows starts[b] .. starts[b + 1] - 1 of q [T, H, d] are the new tokens of
sequence b and the last of its lengths[b] context tokens.  Token j of sequence b
lies in page page_table[b, j // page_size], slot j % page_size, of k_pages and
v_pages [pages, Hkv, page_size, d].  A sequence may have no new tokens; rows before
starts[0] and from starts[S] on are left as they were.  Sequences may share pages (a common prefix)
as long as no call writes a slot twice.
"""

from __future__ import annotations

import ctypes
from typing import Tuple

import torch

from . import layer
from .binding import lib
from .rotary import RotaryParams


class PagedParams(ctypes.Structure):
    """Mirror of ``elsaa_paged_params``."""
    _fields_ = [(n, ctypes.c_int32) for n in ("seqs", "rows", "H", "Hkv", "d", "dtype",
                                              "page_size", "pages", "table_width", "window",
                                              "sinks")] + [("scale", ctypes.c_float)]

    @classmethod
    def make(cls, seqs, rows, H, Hkv, d, dtype, page_size, pages, table_width, window=0, sinks=0,
             scale=0.0) -> "PagedParams":
        return cls(seqs, rows, H, Hkv, d, layer.dtype_code(dtype), page_size, pages, table_width,
                   window, sinks, float(scale))


def validate(p: PagedParams) -> int:
    return lib().elsaa_paged_validate(ctypes.byref(p))


def workspace_bytes(p: PagedParams) -> int:
    return lib().elsaa_paged_workspace_bytes(ctypes.byref(p))


def alloc_workspace(p: PagedParams, device) -> torch.Tensor:
    return layer.alloc_workspace(workspace_bytes(p), device)


def alloc_pages(p: PagedParams, device) -> Tuple[torch.Tensor, torch.Tensor]:
    """k_pages and v_pages of a pool (what they hold is not read before it is written)."""
    shape = (p.pages, p.Hkv, p.page_size, p.d)
    dt = layer.torch_dtype(p.dtype)
    return tuple(torch.empty(shape, dtype=dt, device=device) for _ in range(2))


def _cache(p: PagedParams, k_pages, v_pages, page_table, starts, lengths, dev):
    dt = layer.torch_dtype(p.dtype)
    shape = (p.pages, p.Hkv, p.page_size, p.d)
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        layer.check(name, t, shape, dt, dev)
        if not layer.strided(t) or not layer.rows_apart(t):
            raise ValueError(f"{name}: a contiguous last dimension, strides and a start that are "
                             "multiples of 16 bytes, and no two elements in one place")
    return (k_pages, v_pages,
            layer.as_small("page_table", page_table, (p.seqs, p.table_width), torch.int32, dev),
            layer.as_small("starts", starts, (p.seqs + 1,), torch.int32, dev),
            layer.as_small("lengths", lengths, (p.seqs,), torch.int32, dev))


@layer.on_device(2)
def write(p: PagedParams, rp: RotaryParams, q, k, v, table, q_weight, k_weight, k_pages, v_pages,
          page_table, starts, lengths, qo=None, ws=None, stream=None) -> torch.Tensor:
    """qo [T, H, d], the new tokens' queries normed and rotated at their positions; their keys
    (likewise) and values [T, Hkv, d] go into the pages.  ``rp``: H, Hkv, d and dtype as in ``p``."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    q = layer.as_input("q", q, (p.rows, p.H, p.d), dt, dev)
    k = layer.as_input("k", k, (p.rows, p.Hkv, p.d), dt, dev)
    v = layer.as_input("v", v, (p.rows, p.Hkv, p.d), dt, dev)
    qo = layer.as_output("qo", qo, (p.rows, p.H, p.d), dt, dev, q)
    if rp.rot_dim > 0:
        if table is None:
            raise ValueError("rot_dim > 0 needs a table")
        table = layer.as_small("table", table, (rp.max_pos, rp.rot_dim // 2, 2), torch.float32, dev)
    q_weight = layer.as_small("q_weight", q_weight, (p.d,), torch.float32, dev)
    k_weight = layer.as_small("k_weight", k_weight, (p.d,), torch.float32, dev)
    k_pages, v_pages, page_table, starts, lengths = _cache(p, k_pages, v_pages, page_table,
                                                           starts, lengths, dev)
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p), dev)
    ptr = layer.ptr
    layer.ok("elsaa_paged_write", lib().elsaa_paged_write(
        ctypes.byref(p), ctypes.byref(rp), ptr(q), ptr(k), ptr(v),
        layer.strides_of(2, q, qo, k, v), ptr(table), ptr(q_weight), ptr(k_weight), ptr(qo),
        ptr(k_pages), ptr(v_pages), layer.strides_of(3, k_pages, v_pages), ptr(page_table),
        ptr(starts), ptr(lengths), ptr(ws), ws.numel(), stream))
    return qo


@layer.on_device(1)
def attend(p: PagedParams, q, k_pages, v_pages, page_table, starts, lengths, y=None, ws=None,
           stream=None) -> torch.Tensor:
    """y [T, H, d]: attention of the new tokens q [T, H, d] over their sequences' cached keys and
    values (their own already written)."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    q = layer.as_input("q", q, (p.rows, p.H, p.d), dt, dev)
    y = layer.as_output("y", y, (p.rows, p.H, p.d), dt, dev, q)
    k_pages, v_pages, page_table, starts, lengths = _cache(p, k_pages, v_pages, page_table,
                                                           starts, lengths, dev)
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p), dev)
    ptr = layer.ptr
    layer.ok("elsaa_paged_attend", lib().elsaa_paged_attend(
        ctypes.byref(p), ptr(q), layer.strides_of(2, q, y), ptr(k_pages), ptr(v_pages),
        layer.strides_of(3, k_pages, v_pages), ptr(page_table), ptr(starts), ptr(lengths),
        ptr(y), ptr(ws), ws.numel(), stream))
    return y
