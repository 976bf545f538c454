"""The pages of paged 8-bit caches, shared and moved on the device (the page
entry points ``kv8_*`` of ``include/w4a16.h``).

    refs = kv8_refs(num_pages)                          # all pages free
    kv8_reserve(refs, page_table, seq_lens, added, T)   # pages for new tokens
    kv8_fork(caches, refs, page_table, seq_lens, src, dst)
    kv8_free(refs, page_table, seq_lens, rows, T)
    page_table, refs, used = kv8_compact(caches, refs, page_table, seq_lens)

refs int32 [num_pages] counts the rows of page_table (int32 [B, max_pages])
that hold a page, 0 where it is free; seq_lens int32 [B] is 0 for a row that
holds none.  ``caches`` is a cache (kv8_cache) or a list of them of one size, as
the layers of a model have them: they share refs, page_table and seq_lens.
Nothing is read back to the host, so the calls can be captured in a graph; what
may fail on the device says so in a status tensor (int32 [1]): 0 done, above 0
the pages that were missing, -1 rows that the call refuses; then nothing has
been changed.  Calls that overlap in time must not share a workspace (one per
stream is kept when none is given; a call that is captured finds it there from a
call before, or is given one).
"""

import ctypes

import torch

from . import _here, _lib, _need, _stream
from .kv8 import _cache
from .w8a8 import _empty, _space


def kv8_refs(num_pages, device="cuda"):
    """The counters of a pool whose pages are all free: int32 [num_pages]."""
    return torch.zeros(num_pages, dtype=torch.int32, device=device)


def kv8_pages_workspace_bytes(num_pages, B, n=0):
    """Bytes that kv8_reserve, kv8_fork (of n pairs) and kv8_compact need."""
    size = int(_lib.lib().kv8_pages_workspace_bytes(num_pages, B, n))
    if size < 0:
        raise _lib.W4A16Error("kv8_pages_workspace_bytes: invalid sizes")
    return size


def _caches(caches, refs=None):
    """The caches' arrays as the entry points take them, their count and sizes."""
    if isinstance(caches, dict):
        caches = [caches]
    if not caches:
        raise ValueError("no cache")
    pages, Hkv, T, D, at = _cache(caches[0])
    arrays = list(at)
    for c in caches[1:]:
        *sizes, at = _cache(c)
        if sizes != [pages, Hkv, T, D]:
            raise ValueError("the caches differ in their sizes")
        arrays += at
    if refs is not None:
        _need(refs, torch.int32, "refs", pages)
    return (ctypes.c_void_p * len(arrays))(*arrays), len(caches), pages, T, Hkv, D


def _arrays(caches):
    """One array of each cache (kv8_cache allocates a cache's arrays together)."""
    return [c["k"] for c in ([caches] if isinstance(caches, dict) else caches)]


def _rows(page_table, seq_lens):
    _need(page_table, torch.int32, "page_table")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, width = page_table.shape
    _need(seq_lens, torch.int32, "seq_lens", B)
    return B, width


def _status(status, like, stream):
    if status is None:
        return like.new_empty(1) if stream is None else _empty((1,), torch.int32, like.device, stream)
    _need(status, torch.int32, "status", 1)
    return status


def _call(name, *args):
    status = getattr(_lib.lib(), name)(*args)
    if status:
        _lib.check(status, name)


def kv8_copy_pages(caches, src, dst, stream=None):
    """Copies pages src[i] (int32 [n]) over pages dst[i], codes and scales, in
    every cache.  Pairs with a page out of range are passed over; no dst may be
    named twice or be a src."""
    arrays, count, pages, T, Hkv, D = _caches(caches)
    _need(src, torch.int32, "src")
    _need(dst, torch.int32, "dst", src.numel())
    _here(stream, src, dst, *_arrays(caches))
    _call("kv8_copy_pages", arrays, count, pages, T, Hkv, D, src.data_ptr(), dst.data_ptr(),
          src.numel(), _stream(stream))


def kv8_free(refs, page_table, seq_lens, rows, page_size, stream=None):
    """Gives back the pages of table rows rows (int32 [n]): their counters go
    down, their entries become -1 and their lengths 0.  A row out of range is
    passed over, one named twice is given back once."""
    _need(refs, torch.int32, "refs")
    B, width = _rows(page_table, seq_lens)
    _need(rows, torch.int32, "rows")
    _here(stream, refs, page_table, seq_lens, rows)
    _call("kv8_free", refs.data_ptr(), refs.numel(), page_size, page_table.data_ptr(), width,
          seq_lens.data_ptr(), B, rows.data_ptr(), rows.numel(), _stream(stream))


def kv8_reserve(refs, page_table, seq_lens, added, page_size, status=None, workspace=None,
                stream=None):
    """Makes room for added (int32 [B]) more tokens in every row: takes the
    pages they need, the lowest free ones in the order of the rows, and adds
    them to seq_lens, as kv8_append wants it; below 0 drops that many last tokens
    and gives back the pages that this empties; the page that the row then ends in
    keeps the scales and codes (a NaN too) that kv8_append made of the dropped rows
    and those before them: drafts that must not show are appended to a fork.
    Returns the status: 0, the pages that are missing, or -1 where a row would pass
    the table's width, or after dropping would end within a page that other rows
    hold too."""
    _need(refs, torch.int32, "refs")
    B, width = _rows(page_table, seq_lens)
    _need(added, torch.int32, "added", B)
    _here(stream, refs, page_table, seq_lens, added, status, workspace)
    status = _status(status, refs, stream)
    workspace, nbytes = _space(workspace, kv8_pages_workspace_bytes(refs.numel(), B), refs.device,
                               stream)
    _call("kv8_reserve", refs.data_ptr(), refs.numel(), page_size, page_table.data_ptr(), width,
          seq_lens.data_ptr(), B, added.data_ptr(), status.data_ptr(), workspace.data_ptr(), nbytes,
          _stream(stream))
    return status


def kv8_fork(caches, refs, page_table, seq_lens, src, dst, status=None, workspace=None,
             stream=None):
    """Makes table row dst[i] (int32 [n]), which must be empty, a copy of row
    src[i]: whole pages are shared, a partly filled last one is copied to a page
    of its own, so that both may append.  Returns the status: 0, the pages that
    are missing, or -1 where a row is out of range, a dst is not empty, named
    twice or a src."""
    arrays, count, pages, T, Hkv, D = _caches(caches, refs)
    B, width = _rows(page_table, seq_lens)
    _need(src, torch.int32, "src")
    n = src.numel()
    _need(dst, torch.int32, "dst", n)
    _here(stream, refs, page_table, seq_lens, src, dst, status, workspace, *_arrays(caches))
    status = _status(status, refs, stream)
    workspace, nbytes = _space(workspace, kv8_pages_workspace_bytes(pages, B, n), refs.device,
                               stream)
    _call("kv8_fork", arrays, count, pages, T, Hkv, D, refs.data_ptr(), page_table.data_ptr(),
          width, seq_lens.data_ptr(), B, src.data_ptr(), dst.data_ptr(), n, status.data_ptr(),
          workspace.data_ptr(), nbytes, _stream(stream))
    return status


def kv8_compact(caches, refs, page_table, seq_lens, page_table_out=None, refs_out=None,
                workspace=None, stream=None):
    """Moves the pages in use together at the beginning of the pool: of `used`
    pages in use, those from `used` on go to the free ones below, both in
    ascending order.  Returns (page_table, refs, used int32 [1]) as they are
    then: new tensors, or page_table_out and refs_out, which may be page_table
    and refs themselves.  The pages moved from keep their bytes, so work that
    still goes by the old table stays right until they are taken again."""
    arrays, count, pages, T, Hkv, D = _caches(caches, refs)
    B, width = _rows(page_table, seq_lens)
    _here(stream, refs, page_table, seq_lens, page_table_out, refs_out, workspace,
          *_arrays(caches))
    device = refs.device
    if page_table_out is None:
        page_table_out = _empty((B, width), torch.int32, device, stream)
    _need(page_table_out, torch.int32, "page_table_out", B * width)
    if refs_out is None:
        refs_out = _empty((pages,), torch.int32, device, stream)
    _need(refs_out, torch.int32, "refs_out", pages)
    used = _empty((1,), torch.int32, device, stream)
    workspace, nbytes = _space(workspace, kv8_pages_workspace_bytes(pages, B), device, stream)
    _call("kv8_compact", arrays, count, pages, T, Hkv, D, refs.data_ptr(), refs_out.data_ptr(),
          page_table.data_ptr(), page_table_out.data_ptr(), width, seq_lens.data_ptr(), B,
          used.data_ptr(), workspace.data_ptr(), nbytes, _stream(stream))
    return page_table_out, refs_out, used
