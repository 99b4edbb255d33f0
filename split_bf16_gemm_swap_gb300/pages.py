"""ctypes binding of the page operators in ``include/lowm_pages.h``.

A cache's pages are counted and handed out on the device: :func:`fork_pages`,
:func:`extend_pages`, :func:`compact_pages` and :func:`copy_pages` launch and
return, in the manner of :mod:`.layer`, and wait for nothing.  A page table is
int32 [rows, width]; ``lens`` int32 [rows] says how many tokens each row has;
``refs`` int32 [num_pages] how many rows list a page (0: free).
"""
from __future__ import annotations

import array
import ctypes

import torch

from . import layer
from .layer import _cuda, _current_device, _current_stream, _dense, _i, _l, _launch, _on, _p, _refuse, _row_stride, _rows, _z, function
from .lowm import LOWM_OK, LowmError

# Exported C functions, in header order.
ABI_FUNCTIONS = (
    "lowm_fork_pages",
    "lowm_extend_pages",
    "lowm_extend_pages_workspace",
    "lowm_compact_pages",
    "lowm_compact_pages_workspace",
    "lowm_copy_pages",
)

layer._ARGTYPES.update({
    "lowm_fork_pages": [_p, _l, _p, _i, _p, _i, _i, _p, _i, _i, _p, _l, _p, _p, _p, _p, _p],
    "lowm_extend_pages": [_p, _l, _p, _i, _i, _p, _i, _p, _i, _i, _p, _p, _p, _p, _z, _p],
    "lowm_extend_pages_workspace": [_i],
    "lowm_compact_pages": [_p, _l, _p, _i, _i, _p, _i, _i, _p, _p, _p, _p, _z, _p],
    "lowm_compact_pages_workspace": [_i],
    "lowm_copy_pages": [_p, _i, _p, _p, _i, _i, _p],
})


class lowm_page_span_t(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64)]


def lowm_fork_pages(*args) -> int:
    return function("lowm_fork_pages")(*args)


def lowm_extend_pages(*args) -> int:
    return function("lowm_extend_pages")(*args)


def lowm_extend_pages_workspace(num_pages: int) -> int:
    return function("lowm_extend_pages_workspace")(num_pages)


def lowm_compact_pages(*args) -> int:
    return function("lowm_compact_pages")(*args)


def lowm_compact_pages_workspace(num_pages: int) -> int:
    return function("lowm_compact_pages_workspace")(num_pages)


def lowm_copy_pages(*args) -> int:
    return function("lowm_copy_pages")(*args)


def _table(page_table, lens, refs, device: int):
    """Checks of a table, its lengths and the counts; (rows, width, stride, num_pages)."""
    shape, counted = page_table.shape, refs.shape
    if len(shape) != 2 or len(counted) != 1:
        raise ValueError("page_table must be [rows, width] and refs [num_pages]")
    rows, width = shape
    stride = _row_stride(page_table, "page_table", torch.int32, shape, device)
    _dense(lens, "lens", torch.int32, (rows,), device)
    _dense(refs, "refs", torch.int32, counted, device)
    return rows, width, stride, counted[0]


def _ints(device: int, *sizes, dtype=torch.int32):
    """A tensor of each size (views of one tensor that goes out of sight take the host four times as long)."""
    on = torch.device("cuda", device)
    return [torch.empty(n, dtype=dtype, device=on) for n in sizes]


def fork_pages(page_table, lens, parents, refs, page_size: int, *, out=None, stream=None):
    """Rows that continue others (beam search, sampling several answers), begin empty, or end.

    Row i of the result continues row ``parents[i]`` (int32; negative: empty); rows
    that nobody continues are given up.  Whole pages are shared; an unfinished last
    page stays with the first of its rows, and the others get one of their own, to
    be copied (:func:`copy_pages`).  Returns ``(table, lens, src, dst, missing)``:
    the new rows, the copies (int32 [rows], -1: none) and an int32 [1] count of
    pages that were not to be had.  refs is updated in place; ``out`` is memory for
    the new table, none of it the old one's.
    """
    device = _cuda(page_table, "page_table")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return fork_pages(page_table, lens, parents, refs, page_size, out=out)
    rows, width, stride, num_pages = _table(page_table, lens, refs, device)
    if parents.dim() != 1:
        raise ValueError("parents must be [rows]")
    new_rows = parents.shape[0]
    _dense(parents, "parents", torch.int32, parents.shape, device)
    new_lens, src, dst, missing = _ints(device, new_rows, new_rows, new_rows, 1)
    if out is None:
        out = torch.empty((new_rows, width), dtype=torch.int32, device=page_table.device)
    elif out.data_ptr() == page_table.data_ptr() and out.numel():
        raise ValueError("out must not be page_table itself")
    out_stride = _row_stride(out, "out", torch.int32, (new_rows, width), device)
    s = function("lowm_fork_pages")(
        page_table.data_ptr(), stride, lens.data_ptr(), rows, parents.data_ptr(), new_rows, width, refs.data_ptr(), num_pages,
        page_size, out.data_ptr(), out_stride, new_lens.data_ptr(), src.data_ptr(), dst.data_ptr(), missing.data_ptr(),
        _current_stream(device))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_fork_pages")
    return out, new_lens, src, dst, missing


def extend_pages(page_table, lens, cu_new, refs, page_size: int, tokens: int, *, stream=None):
    """Room for `tokens` new tokens, ``cu_new[b + 1] - cu_new[b]`` (int32 [rows + 1]) of them in row b.

    page_table, lens and refs are updated in place.  Returns ``(positions, slots,
    missing)`` for :func:`.layer.rope_append`: int64 [tokens] each, and an int32 [1]
    count of pages that were not to be had (their tokens have slot -1), among them
    those of rows that :func:`fork_pages` left on another's unfinished page.
    """
    device = _cuda(page_table, "page_table")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return extend_pages(page_table, lens, cu_new, refs, page_size, tokens)
    rows, width, stride, num_pages = _table(page_table, lens, refs, device)
    _dense(cu_new, "cu_new", torch.int32, (rows + 1,), device)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    positions, slots = _ints(device, tokens, tokens, dtype=torch.int64)
    missing, = _ints(device, 1)
    _launch("lowm_extend_pages", (
        page_table.data_ptr(), stride, lens.data_ptr(), rows, width, cu_new.data_ptr(), tokens, refs.data_ptr(), num_pages,
        page_size, positions.data_ptr(), slots.data_ptr(), missing.data_ptr()), max(4 * num_pages, 4), device,
        _current_stream(device))
    return positions, slots, missing


def compact_pages(page_table, lens, refs, page_size: int, *, stream=None):
    """Brings the pages in use together at the front of the pool.

    page_table, which is to hold every sequence of the pool, and refs are updated in
    place.  Returns ``(src, dst, used)``: the moves for :func:`copy_pages` (int32
    [num_pages / 2], -1 behind the last) and an int32 [1] count of the pages in use.
    """
    device = _cuda(page_table, "page_table")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return compact_pages(page_table, lens, refs, page_size)
    rows, width, stride, num_pages = _table(page_table, lens, refs, device)
    moves = num_pages // 2
    src, dst, used = _ints(device, moves, moves, 1)
    _launch("lowm_compact_pages", (
        page_table.data_ptr(), stride, lens.data_ptr(), rows, width, refs.data_ptr(), num_pages, page_size, src.data_ptr(),
        dst.data_ptr(), used.data_ptr()), lowm_compact_pages_workspace(num_pages), device, _current_stream(device))
    return src, dst, used


def copy_pages(caches, src, dst, *, stream=None) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` in every tensor of `caches`.

    caches: tensors [num_pages, ...] of any type whose pages are contiguous (keys,
    values and scales of all layers); src, dst int32 [n], pairs with a negative one
    are passed over.  No page may be a destination twice, or a source and a
    destination.
    """
    device = _cuda(src, "src")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return copy_pages(caches, src, dst)
    shape = src.shape
    if len(shape) != 1:
        raise ValueError("src must be [n]")
    _dense(src, "src", torch.int32, shape, device)
    _dense(dst, "dst", torch.int32, shape, device)
    spans = []
    num_pages = caches[0].size(0) if len(caches) and caches[0].dim() else 0
    nbytes = page_bytes = -1                             # of the tensor before, mostly another layer's like it
    for x in caches:
        if x.get_device() != device or x.dim() == 0 or x.shape[0] != num_pages:
            raise ValueError("caches must be on cuda:%d and have one number of pages" % device)
        if x.is_contiguous():
            if x.nbytes != nbytes:
                nbytes = x.nbytes
                page_bytes = nbytes // num_pages if num_pages else 0
            spans += (x.data_ptr(), page_bytes, page_bytes)
        else:
            if num_pages and not x[0].is_contiguous():
                raise ValueError("the pages of a cache must be contiguous")
            spans += (x.data_ptr(), x.stride(0) * x.element_size(), x[0].nbytes if num_pages else 0)
    held = array.array("q", spans)                       # as lowm_page_span_t lies in memory
    packed = held.buffer_info()[0]
    s = function("lowm_copy_pages")(packed, len(caches), src.data_ptr(), dst.data_ptr(), shape[0], num_pages,
                                    _current_stream(device))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_copy_pages")
