"""Binding of the page entry points of libfa.so: pages of the 8-bit cache copied, shared
between sequences, dealt out and moved together, in every layer of a model.

As in _cache.py, every step runs in the CUDA kernels. A page table is int32 [rows, columns], -1
where a row has no page; refs int32 [num_pages] counts the entries that name each page
(0: free) and starts as zeros beside a table of -1.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from ._cache import _I32, _I64, _SZ, KVCache, _done, _ints, _matrix, _on, _raw_stream
from ._lib import _I, _P, SIGNATURES, lib


class PageTableStruct(ctypes.Structure):
    """fa_page_table of include/fa.h."""
    _fields_ = [("entries", _P), ("stride", _I64), ("rows", _I), ("width", _I), ("refs", _P), ("num_pages", _I), ("page_size", _I)]


_CACHES = _TABLE = ctypes.c_char_p  # a host array of fa_cache, a fa_page_table, as bytes
_PACK = struct.Struct("@PqiiPii")    # PageTableStruct
assert _PACK.size == ctypes.sizeof(PageTableStruct)
SIGNATURES["fa_cache_copy"] = (_I, [_CACHES, _I, _P, _P, _I, _P])
SIGNATURES["fa_cache_fork"] = (_I, [_TABLE, _P, _P, _P])
SIGNATURES["fa_cache_reserve_workspace_bytes"] = (_SZ, [_I, _I, _I])
SIGNATURES["fa_cache_reserve"] = (_I, [_CACHES, _I, _TABLE, _P, _P, _I32, _P, _P, _SZ, _P])
SIGNATURES["fa_cache_compact_workspace_bytes"] = (_SZ, [_I])
SIGNATURES["fa_cache_compact"] = (_I, [_CACHES, _I, _TABLE, _P, _P, _P, _SZ, _P])


def _layers(caches):
    """One KVCache or a sequence of them as the C calls take them: structs, their number, the
    first one."""
    if isinstance(caches, KVCache):
        return caches._bytes, 1, caches
    try:
        caches = list(caches)
        structs = b"".join([c._bytes for c in caches])
    except (TypeError, AttributeError):
        caches = []
    if not caches:
        raise ValueError("caches must be a KVCache or a sequence of them, one for each layer")
    first = caches[0]
    index = first._index
    for c in caches:
        if c._index != index:
            raise ValueError("the layers' caches are on different devices")
    return structs, len(caches), first


def _table(t, refs, page_size, index):
    """The fa_page_table of a table and its counts, the table's rows and columns, and the pages."""
    entries, stride, rows, width = _matrix(t, "page_table", index)
    counts = _ints(refs, "refs", index, None)
    pages = refs.numel()
    if not -2 ** 31 <= page_size < 2 ** 31 or pages >= 2 ** 31:  # others the library refuses
        raise ValueError("page_size and the values of refs must be numbers of 32 bits")
    return _PACK.pack(entries, stride, rows, width, counts, pages, page_size), rows, width, pages


def _maybe(t, what, index, n):
    return None if t is None else _ints(t, what, index, n)


def _workspace(workspace, need, dev):
    """The caller's workspace, or a new one, and its bytes."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev.index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the tensors' device")
    return workspace, workspace.numel() * workspace.element_size()


def _rows_out(t, n, what, dev):
    if t is None:
        return torch.empty(n, dtype=torch.int32, device=dev)
    _ints(t, what, dev.index, n)
    return t


def cache_copy(caches, src, dst, stream=None) -> None:
    """Copies page src[i] to page dst[i], codes and scales, in every layer's cache (fa_cache_copy): int32
    [n] on the device; moves with -1 in either are left out. No page of dst may be another move's
    source or destination."""
    s, n, first = _layers(caches)
    _on(_copy, first.device, stream, s, n, first._index, src, dst)


def _copy(s, layers, index, src, dst):
    a = _ints(src, "src", index, None)
    n = src.numel()
    _done(lib().fa_cache_copy(s, layers, a, _ints(dst, "dst", index, n), n, _raw_stream(index)), "fa_cache_copy")


def cache_fork(page_table, refs, page_size: int, parent=None, keep=None, stream=None) -> None:
    """Rows of page_table become copies of other rows, all at once, in place (fa_cache_fork): row b
    takes the pages of row parent[b] (-1: none, b: its own), of which those of the first keep[b]
    tokens stay (None: all). refs follows, so rows that finish or are cut short give their pages back.
    parent, keep: int32 [rows], one of them at least. Before a row writes into a page that it
    shares, cache_reserve gives it its own."""
    if not isinstance(page_table, torch.Tensor) or not page_table.is_cuda:
        raise ValueError("page_table must be a CUDA tensor")
    _on(_fork, page_table.device, stream, page_table, refs, int(page_size), parent, keep)


def _fork(page_table, refs, page_size, parent, keep):
    index = page_table.get_device()
    t, rows, _, _ = _table(page_table, refs, page_size, index)
    if parent is None and keep is None:
        raise ValueError("give parent, keep or both")
    _done(lib().fa_cache_fork(t, _maybe(parent, "parent", index, rows), _maybe(keep, "keep", index, rows), _raw_stream(index)), "fa_cache_fork")


def cache_reserve_workspace_bytes(cache: KVCache, rows: int, pages: int) -> int:
    """Workspace bytes of cache_reserve for a page table of `rows` rows and `pages` columns."""
    return lib().fa_cache_reserve_workspace_bytes(rows, pages, cache.k.shape[0])


def cache_reserve(caches, page_table, refs, start, count, ok=None, workspace=None, stream=None):
    """Gives row b a page of its own for each of the tokens start[b] + n, n < count[b], that are to be
    written (fa_cache_reserve): free pages, the lowest first, where it has none; a copy, in every
    layer, of a page that it shares and that holds earlier tokens of it. start: int32 [rows] or None for 0; count: int32
    [rows] or one number for every row. Returns ok, int32 [rows]: 0 where pages ran out or the
    tokens pass the table's width; such rows must not be written to. `workspace`: uint8 of
    cache_reserve_workspace_bytes(...) bytes, allocated here if None."""
    s, n, first = _layers(caches)
    return _on(_reserve, first.device, stream, s, n, first, page_table, refs, start, count, ok, workspace)


def _reserve(s, layers, first, page_table, refs, start, count, ok, workspace):
    dev, index = first.device, first._index
    t, rows, width, pages = _table(page_table, refs, first.page_size, index)
    tokens = 0
    if not isinstance(count, torch.Tensor):
        if count is None or not 0 <= int(count) < 2 ** 31:
            raise ValueError("count must be int32 [rows] or a number of tokens")
        tokens, count = int(count), None
    b, c = _maybe(start, "start", index, rows), _maybe(count, "count", index, rows)
    ok = _rows_out(ok, rows, "ok", dev)
    L = lib()
    workspace, have = _workspace(workspace, L.fa_cache_reserve_workspace_bytes(rows, width, pages) if workspace is None else 0, dev)
    _done(L.fa_cache_reserve(s, layers, t, b, c, tokens, ok.data_ptr(), workspace.data_ptr(), have, _raw_stream(index)), "fa_cache_reserve")
    return ok


def cache_compact_workspace_bytes(cache: KVCache) -> int:
    """Workspace bytes of cache_compact."""
    return lib().fa_cache_compact_workspace_bytes(cache.k.shape[0])


def cache_compact(caches, page_table, refs, where=None, live=None, workspace=None, stream=None):
    """Moves the pages in use to the lowest numbers, in every layer, in page_table and in refs
    (fa_cache_compact). Returns where, int32 [num_pages]: each page's new number, -1 for free ones (for other
    tables that name pages), and live, int32 [1]: the pages in use. `workspace`: uint8 of
    cache_compact_workspace_bytes(...) bytes, allocated here if None."""
    s, n, first = _layers(caches)
    return _on(_compact, first.device, stream, s, n, first, page_table, refs, where, live, workspace)


def _compact(s, layers, first, page_table, refs, where, live, workspace):
    dev, index = first.device, first._index
    t, _, _, pages = _table(page_table, refs, first.page_size, index)
    where, live = _rows_out(where, pages, "where", dev), _rows_out(live, 1, "live", dev)
    L = lib()
    workspace, have = _workspace(workspace, L.fa_cache_compact_workspace_bytes(pages) if workspace is None else 0, dev)
    _done(L.fa_cache_compact(s, layers, t, where.data_ptr(), live.data_ptr(), workspace.data_ptr(), have, _raw_stream(index)),
          "fa_cache_compact")
    return where, live
