"""Pages of a paged cache: a pool on the device from which sequences reserve, fork and release
them, copies of pages, and compaction of a cache in place (see the sections on them in
include/up.h).

    pool = PagePool.full(num_pages)                     # all pages free, tables of -1
    reserve_pages(pool, table, page_size, old_lens, new_lens)
    table2, lens2, copies = fork_pages(pool, table, lens, page_size, parents)
    copy_pages(cache, copies)                           # for every layer's cache
    new_lens = compact_kv(cache, cu_seqlens, keep)      # for every layer's cache
    release_pages(pool, table, page_size, new_lens, old_lens)
"""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from .paged import PagedKV, _error, _int32, _L, _need, _on, _raw


class _CPool(ctypes.Structure):
    """up_page_pool of include/up.h."""
    _fields_ = [("refs", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("num_free", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64)]


class PagePool:
    """The pages that block tables share out: refs int32 [num_pages] (entries that hold each page),
    free_pages int32 [num_pages] (a stack of the free ones) and num_free int32 [1].  Holds
    the tensors; calls change their contents in place."""

    __slots__ = ("refs", "free_pages", "num_free", "num_pages", "device", "struct", "ref")

    def __init__(self, refs, free_pages, num_free):
        _need(refs, "refs", torch.int32, None)
        if refs.dim() != 1:
            raise ValueError("refs must be [num_pages]")
        dev = refs.device
        _need(free_pages, "free_pages", torch.int32, dev, refs.shape)
        _need(num_free, "num_free", torch.int32, dev, (1,))
        c = _CPool(refs.data_ptr(), free_pages.data_ptr(), num_free.data_ptr(), refs.numel())
        for put, x in zip(_PUT, (refs, free_pages, num_free, refs.numel(), dev, c, ctypes.byref(c))):
            put(self, x)

    @classmethod
    def full(cls, num_pages, device="cuda"):
        """A pool whose pages are all free, page 0 on top."""
        if num_pages < 1:
            raise ValueError("num_pages must be positive")
        i = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        return cls(torch.zeros_like(i), i, torch.full((1,), num_pages, dtype=torch.int32, device=device))

    def _fixed(self, name, value=None):
        raise AttributeError(f"{name}: a PagePool's attributes are fixed")

    __setattr__ = __delattr__ = _fixed

    def __reduce__(self):  # copies get a struct of their own
        return type(self), (self.refs, self.free_pages, self.num_free)

    def __repr__(self):
        return f"PagePool({self.num_pages} pages on {self.device})"


_PUT = tuple(PagePool.__dict__[name].__set__ for name in PagePool.__slots__)


def _table(pool, block_table, page_size):
    """Rows and width of a block table of the pool's, and the page size as a C int."""
    if not isinstance(pool, PagePool):
        raise TypeError("pool must be a PagePool")
    _need(block_table, "block_table", torch.int32, pool.device)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [num_seqs, max_pages]")
    return (*block_table.shape, _int32(operator.index(page_size)))


def reserve_pages(pool, block_table, page_size, have, want, stream=None):
    """Gives free pages to the entries of block_table int32 [num_seqs, max_pages] that the tokens
    have[s] .. want[s] - 1 (int32 [num_seqs] each) begin and that hold none (see up_reserve_pages)."""
    B, mp, ps = _table(pool, block_table, page_size)
    _need(have, "have", torch.int32, pool.device, (B,))
    _need(want, "want", torch.int32, pool.device, (B,))
    st = _L().up_reserve_pages(pool.ref, block_table.data_ptr(), B, mp, ps, have.data_ptr(), want.data_ptr(),
                               _raw(stream, pool.device))
    if st:
        raise _error("up_reserve_pages", st)


def release_pages(pool, block_table, page_size, first, end, stream=None):
    """Lets go of the pages that begin in the tokens first[s] .. end[s] - 1 of each sequence (int32
    [num_seqs]; first None: 0); their entries become -1 (see up_release_pages)."""
    B, mp, ps = _table(pool, block_table, page_size)
    if first is not None:
        _need(first, "first", torch.int32, pool.device, (B,))
    _need(end, "end", torch.int32, pool.device, (B,))
    st = _L().up_release_pages(pool.ref, block_table.data_ptr(), B, mp, ps,
                               None if first is None else first.data_ptr(), end.data_ptr(), _raw(stream, pool.device))
    if st:
        raise _error("up_release_pages", st)


def fork_pages(pool, block_table, kv_lens, page_size, parents, table_out=None, lens_out=None, copies=None,
               stream=None):
    """Copies of the sequences parents int32 [children] of block_table [num_seqs, max_pages] and
    kv_lens [num_seqs]: returns (table_out [children, max_pages], lens_out [children], copies
    [3, children]), all int32.  Full pages are shared; copies, for copy_pages, says what
    the children's own last pages take over (see up_fork_pages)."""
    B, mp, ps = _table(pool, block_table, page_size)
    dev = pool.device
    _need(kv_lens, "kv_lens", torch.int32, dev, (B,))
    _need(parents, "parents", torch.int32, dev)
    if parents.dim() != 1:
        raise ValueError("parents must be [children]")
    n = parents.numel()
    with _on(stream):
        if table_out is None:
            table_out = torch.empty((n, mp), dtype=torch.int32, device=dev)
        else:
            _need(table_out, "table_out", torch.int32, dev, (n, mp))
        if lens_out is None:
            lens_out = torch.empty(n, dtype=torch.int32, device=dev)
        else:
            _need(lens_out, "lens_out", torch.int32, dev, (n,))
        if copies is None:
            copies = torch.empty((3, n), dtype=torch.int32, device=dev)
        else:
            _need(copies, "copies", torch.int32, dev, (3, n))
        st = _L().up_fork_pages(pool.ref, block_table.data_ptr(), kv_lens.data_ptr(), B, mp, ps, parents.data_ptr(),
                                n, table_out.data_ptr(), lens_out.data_ptr(), copies.data_ptr(), _raw(stream, dev))
    if st:
        raise _error("up_fork_pages", st)
    return table_out, lens_out, copies


def copy_pages(cache, copies, stream=None):
    """Copies rows of pages of a PagedKV's keys, values and positions: copies int32 [3, n] holds
    the source pages, the destination pages and the rows (see up_copy_pages)."""
    if not isinstance(cache, PagedKV):
        raise TypeError("cache must be a PagedKV")
    _need(copies, "copies", torch.int32, cache.device)
    if copies.dim() != 2 or copies.shape[0] != 3:
        raise ValueError("copies must be [3, n]")
    st = _L().up_copy_pages(cache.ref, copies.data_ptr(), copies.shape[1], _raw(stream, cache.device))
    if st:
        raise _error("up_copy_pages", st)


@functools.lru_cache(maxsize=256)
def compact_kv_workspace(max_tokens, num_seqs, Hk, d) -> int:
    """Bytes of compact_kv's workspace (0: sizes it does not take)."""
    return int(_L().up_compact_kv_workspace(max_tokens, num_seqs, Hk, d))


def compact_kv(cache, cu_seqlens, keep, cu_blocks=None, G=1, max_tokens=None, kv_lens_out=None, workspace=None,
               stream=None):
    """Compacts a PagedKV in place: of each sequence's last cu_seqlens[s+1] - cu_seqlens[s] cached
    tokens those whose flag in keep (uint8, one for G tokens, a sequence's from cu_blocks[s] on) is
    set move together behind the tokens before them; returns the lengths that remain, int32
    [num_seqs] (see up_compact_kv).

    max_tokens: what cu_seqlens[num_seqs] is at most (default: what keep's flags stand for, as far as the
    block table goes); kv_lens_out may be the cache's own kv_lens, but where several layers' caches share
    them in the last layer's call only: the other layers still need the old lengths."""
    if not isinstance(cache, PagedKV):
        raise TypeError("cache must be a PagedKV")
    dev, B = cache.device, cache.num_seqs
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, (B + 1,))
    _need(keep, "keep", torch.uint8, dev)
    if cu_blocks is not None:
        _need(cu_blocks, "cu_blocks", torch.int32, dev, (B + 1,))
    G = _int32(operator.index(G))
    if max_tokens is None:
        # (tokens may be more than the pool's slots: sequences share pages, and let some go)
        max_tokens = min(keep.numel() * max(G, 1), cache.block_table.numel() * cache.page_size, 2 ** 31 - 1)
    T = max(-1, min(operator.index(max_tokens), 2 ** 62))
    with _on(stream):
        if kv_lens_out is None:
            kv_lens_out = torch.empty(B, dtype=torch.int32, device=dev)
        elif kv_lens_out is not cache.kv_lens:
            _need(kv_lens_out, "kv_lens_out", torch.int32, dev, (B,))
        if workspace is None:
            size = compact_kv_workspace(T, B, cache.Hk, cache.d)
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        else:
            if not isinstance(workspace, torch.Tensor):
                raise TypeError("workspace must be a torch.Tensor")
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace must be contiguous and on {dev}")
            size = workspace.numel() * workspace.element_size()
        st = _L().up_compact_kv(cache.ref, cu_seqlens.data_ptr(), T, keep.data_ptr(), keep.numel(),
                                None if cu_blocks is None else cu_blocks.data_ptr(), G, kv_lens_out.data_ptr(),
                                workspace.data_ptr(), size, _raw(stream, dev))
    if st:
        raise _error("up_compact_kv", st)
    return kv_lens_out
