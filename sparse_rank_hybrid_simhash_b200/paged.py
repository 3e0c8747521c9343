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
from .rotary import RotaryParams, angles_and_weights


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


def _cache(p: PagedParams, k_pages, v_pages, page_table, starts, lengths, dt, dev):
    shape = (p.pages, p.Hkv, p.page_size, p.d)
    return (layer.place(dev, 3, ("k_pages", k_pages, shape, dt, layer.as_output),
                        ("v_pages", v_pages, shape, dt, layer.as_output)),
            layer.place(dev, 0, ("page_table", page_table, (p.seqs, p.table_width), torch.int32,
                                 layer.as_small),
                        ("starts", starts, (p.seqs + 1,), torch.int32, layer.as_small),
                        ("lengths", lengths, (p.seqs,), torch.int32, layer.as_small)))


@layer.on_device(2)
def write(p: PagedParams, rp: RotaryParams, q, k, v, table, q_weight, k_weight, k_pages, v_pages,
          page_table, starts, lengths, qo=None, ws=None, stream=None) -> torch.Tensor:
    """qo [T, H, d], the new tokens' queries normed and rotated at their positions; their keys
    (likewise) and values [T, Hkv, d] go into the pages.  ``rp``: H, Hkv, d and dtype as in ``p``."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    sq, sk = (p.rows, p.H, p.d), (p.rows, p.Hkv, p.d)
    if qo is None:
        qo = layer.like(q)
    (pq, pqo, pk, pv), strides, _held = layer.place(
        dev, 2, ("q", q, sq, dt, layer.as_input), ("qo", qo, sq, dt, layer.as_output),
        ("k", k, sk, dt, layer.as_input), ("v", v, sk, dt, layer.as_input))
    (ptable, pwq, pwk), _small = angles_and_weights(rp, table, q_weight, k_weight, dev)
    ((pkp, pvp), page_strides, _), ((ppt, pst, plen), _, _rows) = _cache(
        p, k_pages, v_pages, page_table, starts, lengths, dt, dev)
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p), dev)
    layer.ok("elsaa_paged_write", lib().elsaa_paged_write(
        ctypes.byref(p), ctypes.byref(rp), pq, pk, pv, strides, ptable, pwq, pwk, pqo, pkp, pvp,
        page_strides, ppt, pst, plen, ws.data_ptr(), ws.numel(), stream))
    return qo


@layer.on_device(1)
def attend(p: PagedParams, q, k_pages, v_pages, page_table, starts, lengths, y=None, ws=None,
           stream=None) -> torch.Tensor:
    """y [T, H, d]: attention of the new tokens q [T, H, d] over their sequences' cached keys and
    values (their own already written)."""
    dev, dt = q.device, layer.torch_dtype(p.dtype)
    sq = (p.rows, p.H, p.d)
    if y is None:
        y = layer.like(q)
    (pq, py), strides, _held = layer.place(dev, 2, ("q", q, sq, dt, layer.as_input),
                                           ("y", y, sq, dt, layer.as_output))
    ((pkp, pvp), page_strides, _), ((ppt, pst, plen), _, _rows) = _cache(
        p, k_pages, v_pages, page_table, starts, lengths, dt, dev)
    ws = layer.as_workspace(ws, lambda: workspace_bytes(p), dev)
    layer.ok("elsaa_paged_attend", lib().elsaa_paged_attend(
        ctypes.byref(p), pq, strides, pkp, pvp, page_strides, ppt, pst, plen, py, ws.data_ptr(),
        ws.numel(), stream))
    return y
