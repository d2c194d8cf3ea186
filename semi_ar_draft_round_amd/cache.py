"""The paged key/value cache of a serving process, over the C ABI.

PagedCache owns the device buffers of include/dspark_cache.h (the pools of all
layers, the page table and its bookkeeping, every output of the page calls)
and calls the entry points in the order a round needs:

    ell = cache.reserve(d.ell, gamma)             # after dspark_schedule
    for layer in ...:
        q = cache.append(layer, q, k, v, ...)     # norms, rotation, pages
        o, _ = cache.attend(layer, q, ...)
    cache.commit(d.n_acc)                         # after dspark_verify

Nothing is allocated after construction except output tensors and the
attention's workspace where the caller does not pass them, from torch's
allocator, so a round can be captured in a HIP graph.  All calls run on the
current stream.
"""

from __future__ import annotations

import torch

from . import binding as B


class PagedCache:
    def __init__(self, layers: int, slots: int, max_tokens: int, n_pages: int, heads_kv: int, dim: int, page: int = 64,
                 fmt: int = B.CACHE_BF16, window: int = 0, sinks: int = 0, device="cuda:0"):
        """slots: requests; max_tokens: the longest a request may get (its
        rows of a round included); window, sinks: the attention's (0: none),
        so that commit can release what no later row sees."""
        dev = torch.device(device)
        nb = B.dspark_cache_page_bytes(fmt, heads_kv, dim, page)
        if nb == 0 or layers < 1 or slots < 1 or max_tokens < 1 or n_pages < 1:
            raise ValueError(f"no cache of {layers} layers, {slots} slots, {max_tokens} tokens, {n_pages} pages of "
                             f"{page} tokens, {heads_kv} heads of {dim}, format {fmt}")
        if not 0 <= window <= 0x7FFFFFFF or not 0 <= sinks <= 0x7FFFFFFF:
            raise ValueError("window and sinks must be 0 .. 2^31 - 1")
        self.heads_kv, self.dim, self.page, self.fmt = heads_kv, dim, page, fmt
        self.window, self.sinks = window, sinks
        i32 = dict(dtype=torch.int32, device=dev)
        max_pages = -(-max_tokens // page)
        self.pool = torch.empty((layers, n_pages, nb), dtype=torch.uint8, device=dev)
        self.table = torch.empty((slots, max_pages), **i32)
        self.length = torch.empty(slots, **i32)
        self.ref = torch.empty(n_pages, **i32)
        self.bits = torch.empty((n_pages + 31) // 32, **i32)
        # outputs of reserve and compact
        self.ell = torch.full((slots,), -1, **i32)
        self.status = torch.zeros(1, **i32)
        self.pairs = torch.empty((max(slots, n_pages // 2), 2), **i32)
        self.n_pairs = torch.zeros(1, **i32)
        kinds = (B.CACHE_WS_RESERVE, B.CACHE_WS_FORK, B.CACHE_WS_COMPACT)
        self.ws = torch.empty(max(1, *(B.dspark_cache_workspace_size(k, slots, 0, max_pages, n_pages) for k in kinds)),
                              dtype=torch.uint8, device=dev)
        self.gamma = 0
        self.reset()

    def reset(self):
        B.dspark_cache_reset(self.table, self.length, self.ref, self.bits)

    def reserve(self, ell, gamma: int):
        """Pages for every request's ell[r] + 1 rows (-1: none), shared pages
        that will be written copied.  Returns ell as granted (-1 where the
        pages ran out; self.status then reads binding.ENOPAGES), which the
        round's append, attend and commit use."""
        self.gamma = gamma
        B.dspark_cache_reserve(self.table, self.length, self.ref, self.bits, ell, gamma, page=self.page,
                               ell_out=self.ell, pairs=self.pairs[:self.table.shape[0]], n_pairs=self.n_pairs,
                               status=self.status, ws=self.ws)
        B.dspark_cache_copy(self.pool, self.pairs[:self.table.shape[0]], self.n_pairs)
        return self.ell

    def append(self, layer: int, q, k, v, *, wq=None, wk=None, eps=1e-6, freq=None, adjacent=False, row0=None,
               q_out=None):
        """The reserved rows' K and V into layer's pages; returns q with its
        norm and rotation (dspark_cache_append)."""
        return B.dspark_cache_append(q, k, v, self.pool[layer], self.table, self.length, self.ell, self.gamma,
                                     fmt=self.fmt, page=self.page, wq=wq, wk=wk, eps=eps, freq=freq,
                                     adjacent=adjacent, row0=row0, q_out=q_out)

    def attend(self, layer: int, q, *, scale=None, row0=None, out=None, lse=None, ws=None):
        """The reserved rows' attention over layer's pages
        (dspark_cache_attention with the cache's window)."""
        return B.dspark_cache_attention(q, self.pool[layer], self.table, self.length, self.ell, self.gamma,
                                        fmt=self.fmt, page=self.page, heads_kv=self.heads_kv, scale=scale,
                                        window=self.window, sinks=self.sinks, row0=row0, out=out, lse=lse, ws=ws)

    def commit(self, n_acc):
        """Keep the anchor and the first n_acc[r] drafts of the reserved rows."""
        B.dspark_cache_commit(self.table, self.length, self.ref, self.bits, self.ell, n_acc, self.gamma,
                              page=self.page, window=self.window, sinks=self.sinks)

    def fork(self, parent):
        """Request r takes over parent[r]'s tokens, shared (r: stays; -1: empty)."""
        B.dspark_cache_fork(self.table, self.length, self.ref, self.bits, parent, page=self.page, ws=self.ws)

    def compact(self):
        """Pages in use to the low ids of every layer's pool."""
        B.dspark_cache_compact(self.table, self.ref, self.bits, pairs=self.pairs, n_pairs=self.n_pairs, ws=self.ws)
        B.dspark_cache_copy(self.pool, self.pairs, self.n_pairs)

    def read(self, layer: int, T: int, start=None, count=None):
        """k, v [slots][T][heads_kv][dim]: tokens start[r] .. of every request
        (start None: from the first; count None: the committed ones)."""
        if count is None:
            count = self.length if start is None else self.length - start
        return B.dspark_cache_read(self.pool[layer], self.table, start, count, T, fmt=self.fmt, page=self.page,
                                   heads_kv=self.heads_kv, dim=self.dim)
