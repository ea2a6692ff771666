"""Pages of a pool of states: Python binding of ``gla_pages_*`` (``include/gla.h`` has the
contracts). All bookkeeping is int32 on the device; nothing is read back by these calls.

    pool  [P, ...]  P pages (any dtype; a page is a multiple of 16 bytes)
    table [R, M]    the pages of each row, negative where there is none
    free  [P]       stack of free pages, ``count`` [1] of them, the top last

Planning needs a little scratch: a ``workspace`` of the caller's (any type, at least
``pages_workspace_size`` bytes), or the library's own of the stream.
"""
from __future__ import annotations

import torch

from .gla import _check, _addr, _launch, _on_stream, _workspace, load_library
from .hda import _fail, _tensor


def _pool(pool):
    _tensor(pool, "pool")
    if pool.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if pool.dim() < 1 or not pool.is_contiguous():
        raise ValueError("pool must be contiguous, [P, ...]")
    P = pool.shape[0]
    per = 1
    for n in pool.shape[1:]:
        per *= n
    return P, per * pool.element_size()


def _ints(t, name, dev, shape=None):
    _tensor(t, name)
    _check(t, name, torch.int32, (t.numel(),) if shape is None else shape, dev)
    return t


def _book(table, free, count, P, dev):
    _tensor(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be [R, M]")
    _ints(table, "table", dev, table.shape)
    _ints(free, "free", dev, (P,))
    _ints(count, "count", dev, (1,))
    return table.shape


def pages_copy(pool, src, dst, *, stream=None):
    """pool[dst[i]] = pool[src[i]] for every i whose two numbers are not negative."""
    if stream is not None:
        return _on_stream(stream, pages_copy, pool, src, dst)
    lib = load_library()
    P, nb = _pool(pool)
    n = _ints(src, "src", pool.device).numel()
    _ints(dst, "dst", pool.device, (n,))
    rc = _launch(lib.gla_pages_copy, pool.device, _addr(pool), P, nb, _addr(src), _addr(dst), n)
    _fail(lib, rc, "gla_pages_copy")


def pages_workspace_size(table, free, requests: int = 0) -> int:
    """Bytes of workspace that are enough for each of the calls below, with up to ``requests`` parents
    or rows."""
    for t, n in ((table, "table"), (free, "free")):
        _tensor(t, n)
    if table.dim() != 2:
        raise ValueError("table must be [R, M]")
    R, M = table.shape
    return int(load_library().gla_pages_workspace_size(free.numel(), R, M, requests))


def pages_fork(pool, table, free, count, parents, children, *, workspace=None, stream=None):
    """Rows ``children`` become copies of rows ``parents`` on pages taken from the stack."""
    if stream is not None:
        return _on_stream(stream, pages_fork, pool, table, free, count, parents, children,
                          workspace=workspace)
    lib = load_library()
    P, nb = _pool(pool)
    R, M = _book(table, free, count, P, pool.device)
    n = _ints(parents, "parents", pool.device).numel()
    _ints(children, "children", pool.device, (n,))
    rc = _launch(lib.gla_pages_fork_ex, pool.device, _addr(pool), P, nb, _addr(table), R, M,
                 _addr(free), _addr(count), _addr(parents), _addr(children), n,
                 *_workspace(workspace, pool.device))
    _fail(lib, rc, "gla_pages_fork")


def pages_free(table, free, count, rows, *, workspace=None, stream=None):
    """The pages of ``rows`` go back on the stack; the rows have none afterwards."""
    if stream is not None:
        return _on_stream(stream, pages_free, table, free, count, rows, workspace=workspace)
    lib = load_library()
    for t, n in ((table, "table"), (free, "free")):
        _tensor(t, n)
    dev = table.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    P = free.numel()
    R, M = _book(table, free, count, P, dev)
    _ints(rows, "rows", dev)
    rc = _launch(lib.gla_pages_free_ex, dev, P, _addr(table), R, M, _addr(free), _addr(count),
                 _addr(rows), rows.numel(), *_workspace(workspace, dev))
    _fail(lib, rc, "gla_pages_free")


def pages_compact(pool, table, free, count, *, workspace=None, stream=None):
    """The live pages move down to 0 .. n-1; the table follows, the stack is rebuilt."""
    if stream is not None:
        return _on_stream(stream, pages_compact, pool, table, free, count, workspace=workspace)
    lib = load_library()
    P, nb = _pool(pool)
    R, M = _book(table, free, count, P, pool.device)
    rc = _launch(lib.gla_pages_compact_ex, pool.device, _addr(pool), P, nb, _addr(table), R, M,
                 _addr(free), _addr(count), *_workspace(workspace, pool.device))
    _fail(lib, rc, "gla_pages_compact")
