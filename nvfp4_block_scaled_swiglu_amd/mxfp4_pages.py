"""Pages of MXFP4 caches (``include/mxfp4.h``) - Python binding.

Which pages each sequence holds is kept on the device, so that sequences can be lengthened,
forked, cut back and moved without the host waiting for it, also in a captured graph. The
block table and lengths are those that ``mxfp4_cache_append`` and ``mxfp4_attention`` take (rows of
the slots in a batch). Calls, checks, streams and errors are those of ``mxfp4.py``.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

import nvfp4_block_scaled_swiglu_amd as nv

from .mxfp4 import Mxfp4Cache, _buffer, _cache, _CPages, _int32, _MOST, _On


@dataclass
class Mxfp4Pages:
    """Sequences in slots and the pages that they hold: the first ceil(length / page_size) entries
    of a slot's row."""
    block_table: torch.Tensor  # int32 [slots, max_pages]
    seq_lens: torch.Tensor     # int32 [slots]
    refs: torch.Tensor         # int32 [num_pages] entries that hold each page; below 1: free
    page_size: int

    @property
    def num_pages(self) -> int:
        return self.refs.shape[0]


def empty_mxfp4_pages(slots: int, max_pages: int, num_pages: int, page_size: int, device) -> Mxfp4Pages:
    """Empty sequences, every page free."""
    return Mxfp4Pages(torch.full((slots, max_pages), -1, dtype=torch.int32, device=device),
                      torch.zeros((slots,), dtype=torch.int32, device=device),
                      torch.zeros((num_pages,), dtype=torch.int32, device=device), page_size)


def _pages(p: Mxfp4Pages):
    """The record's C form and its tensors."""
    if not isinstance(p, Mxfp4Pages):
        raise ValueError("pages must be an Mxfp4Pages")
    _int32(p.block_table, "pages.block_table", 2)
    _int32(p.seq_lens, "pages.seq_lens", 1)
    _int32(p.refs, "pages.refs", 1)
    slots, pages = p.block_table.shape
    if p.seq_lens.shape[0] != slots:
        raise ValueError("pages.block_table and pages.seq_lens disagree about the slots")
    if not -_MOST <= p.page_size <= _MOST:
        raise ValueError("pages.page_size must fit 64 bits")
    stride = p.block_table.stride(0) if slots > 1 else pages
    return (_CPages(p.block_table.data_ptr(), p.seq_lens.data_ptr(), p.refs.data_ptr(), slots, pages, stride, p.refs.shape[0],
                    p.page_size), (p.block_table, p.seq_lens, p.refs))


def _lists(first, name: str, second=None, other: str = ""):
    _int32(first, name, 1)
    if second is not None and _int32(second, other, 1).shape != first.shape:
        raise ValueError(f"{name} and {other} must have one length")
    return first.shape[0]


def _workspace(on: _On, workspace, size: int):
    """(pointer, bytes) of the caller's workspace or one of `size` bytes, and what keeps it."""
    if workspace is None:
        workspace = torch.empty((max(0, size),), dtype=torch.uint8, device=on.device)
    elif _buffer(workspace, "workspace", 0).device != on.device:
        raise ValueError("workspace must be on the device of the pages")
    else:
        on.use(workspace)
    return workspace


def mxfp4_pages_free(pages: Mxfp4Pages, slots, keep=None, stream=None, strict: Optional[bool] = None) -> Optional[Mxfp4Pages]:
    """Cut the sequences in `slots` (int32 [n]) back to `keep` tokens (int32 [n]; None: none) and give
    back the pages behind them. Returns pages."""
    p, pt = _pages(pages)
    n = _lists(slots, "slots", keep, "keep")
    with _On(stream, *pt, slots, *(() if keep is None else (keep,))) as on:
        if not nv._call("mxfp4_pages_free", p, slots.data_ptr(), None if keep is None else keep.data_ptr(), n, on.handle,
                        strict=strict):
            return None
    return pages


def mxfp4_pages_fork(pages: Mxfp4Pages, parents, children, stream=None, strict: Optional[bool] = None):
    """Make each empty slot children[i] a copy of sequence parents[i] (int32 [n] both), sharing its
    pages. Returns int32 [n]: 1 where that was done."""
    p, pt = _pages(pages)
    n = _lists(parents, "parents", children, "children")
    with _On(stream, *pt, parents, children) as on:
        done = parents.new_empty((n,))
        if not nv._call("mxfp4_pages_fork", p, parents.data_ptr(), children.data_ptr(), n, done.data_ptr(), on.handle,
                        strict=strict):
            return None
    return done


def mxfp4_pages_reserve_workspace_bytes(pages: Mxfp4Pages, n: int) -> int:
    """Bytes of the workspace of a call for n slots; raises ValueError where it would be refused."""
    return _bytes(nv.lib().mxfp4_pages_reserve_workspace_bytes(_pages(pages)[0], max(-1, min(n, 1 << 62))))


def _bytes(size: int) -> int:
    if size < 0:
        raise ValueError(nv.lib().nvfp4_last_error().decode(errors="replace"))
    return int(size)


def mxfp4_pages_reserve(pages: Mxfp4Pages, slots, lens, workspace=None, stream=None, strict: Optional[bool] = None):
    """Lengthen the sequences in `slots` to `lens` tokens (int32 [n] both), with new pages for them.
    Returns (done, src, dst), int32 [n] each: done[i] is 1 where that was possible (also behind entries that there
    were too few pages for, if it needs none), and page src[i], of
    which others hold the beginning too, has to be copied to dst[i] in every cache
    (mxfp4_cache_copy; -1: nothing to copy) before the sequence's next token is written and before
    pages are given out again."""
    p, pt = _pages(pages)
    n = _lists(slots, "slots", lens, "lens")
    with _On(stream, *pt, slots, lens) as on:
        done, src, dst = slots.new_empty((3, n)).unbind()
        workspace = _workspace(on, workspace, nv.lib().mxfp4_pages_reserve_workspace_bytes(p, n) if workspace is None else 0)
        if not nv._call("mxfp4_pages_reserve", p, slots.data_ptr(), lens.data_ptr(), n, done.data_ptr(), src.data_ptr(),
                        dst.data_ptr(), workspace.data_ptr(), workspace.numel(), on.handle, strict=strict):
            return None
    return done, src, dst


def mxfp4_pages_compact_workspace_bytes(pages: Mxfp4Pages) -> int:
    """Bytes of the workspace; raises ValueError where the call would be refused."""
    return _bytes(nv.lib().mxfp4_pages_compact_workspace_bytes(_pages(pages)[0]))


def mxfp4_pages_compact(pages: Mxfp4Pages, out: Optional[Mxfp4Pages] = None, workspace=None, stream=None,
                        strict: Optional[bool] = None):
    """Renumber the used pages so that they are the first ones. Returns (after, src, dst, used): the
    record after it (out, which may be `pages`; by default new, sharing the lengths), the moves for
    mxfp4_cache_copy (int32 [num_pages // 2], -1 behind the last), and how many pages are in use (int32 [1])."""
    p, pt = _pages(pages)
    with _On(stream, *pt) as on:
        if out is None:
            out = Mxfp4Pages(pages.block_table.new_empty((p.slots, p.max_pages)), pages.seq_lens, torch.empty_like(pages.refs),
                             pages.page_size)
            table, stride, refs, lens = out.block_table.data_ptr(), p.max_pages, out.refs.data_ptr(), p.seq_lens
        else:
            o, ot = _pages(out)
            if (o.slots, o.max_pages, o.num_pages, o.page_size) != (p.slots, p.max_pages, p.num_pages, p.page_size):
                raise ValueError("out must be of the size of pages")
            if any(t.device != on.device for t in ot):
                raise ValueError("out must be on the device of pages")
            on.use(*ot)
            table, stride, refs, lens = o.block_table, o.table_stride, o.refs, o.seq_lens
        moves = p.num_pages // 2
        src, dst, used = pages.refs.new_empty((2 * moves + 1,)).split((moves, moves, 1))
        workspace = _workspace(on, workspace, nv.lib().mxfp4_pages_compact_workspace_bytes(p) if workspace is None else 0)
        if not nv._call("mxfp4_pages_compact", p, table, stride, refs, src.data_ptr(), dst.data_ptr(), used.data_ptr(),
                        workspace.data_ptr(), workspace.numel(), on.handle, strict=strict):
            return None
        if lens != p.seq_lens:
            out.seq_lens.copy_(pages.seq_lens)
    return out, src, dst, used


def mxfp4_cache_copy(cache: Mxfp4Cache, src, dst, target: Optional[Mxfp4Cache] = None, stream=None,
                     strict: Optional[bool] = None) -> Optional[Mxfp4Cache]:
    """Copy pages src[i] of the cache to dst[i] (int32 [n] both) of target, by default the same cache;
    pairs with a number out of range are passed over. Returns target."""
    c, ct = _cache(cache)
    t, tt = (c, ()) if target is None or target is cache else _cache(target)
    n = _lists(src, "src", dst, "dst")
    with _On(stream, *ct, *tt, src, dst) as on:
        if not nv._call("mxfp4_cache_copy", c, t, src.data_ptr(), dst.data_ptr(), n, on.handle, strict=strict):
            return None
    return cache if target is None else target
