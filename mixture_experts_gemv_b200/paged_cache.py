"""A paged cache of keys and values for sequences that grow, fork and end.

The tensors of all layers, the block tables and the lengths live on the device, laid out as moe_qk_norm_rope
and moe_attention_decode take them; which page belongs to whom is host bookkeeping:

  open      a row of the block tables for a new sequence
  append    room for new tokens: their positions and slots; a page that the new tokens would write and
            another sequence shares is copied first (moe_copy_pages), so forks are copied on write
  fork      a new row that shares all pages of another
  close     gives a row and its unshared pages back
  compact   moves the live pages to the front of the cache and rewrites the block tables, in one launch,
            so that the pages behind them can be used otherwise

This module is host logic only: the copies run in libmoe's kernels (or, for tests on the CPU, in the ops
object the caller passes). Work is enqueued on the current stream; what reads or writes the cache has to be
ordered with it, as on one stream it is. Not thread-safe.
"""
from __future__ import annotations

import heapq

from ._lib import MOE_ERR_BAD_ARG, MoeError, MoeKvCache, moe_copy_pages


class LibmoeCacheOps:
    """The device work of a cache on a CUDA device."""

    def copy_pages(self, cache, src, dst, block_tables=None):
        moe_copy_pages(cache, src, dst, block_tables=block_tables)


def _refuse(msg: str):
    raise MoeError(MOE_ERR_BAD_ARG, msg)


class PagedKvCache:
    """n_layers caches of num_pages pages of page_size tokens that share their block tables [max_seqs, pages of
    max_tokens] and lengths [max_seqs]. `cache` is the descriptor for the kernels."""

    def __init__(self, n_layers: int, num_pages: int, page_size: int, n_kv: int, head_dim: int, max_seqs: int,
                 max_tokens: int, dtype=None, layout: str = "HND", k_scale: float = 1.0, v_scale: float = 1.0,
                 device="cuda", ops=None):
        import torch
        if min(n_layers, num_pages, page_size, n_kv, head_dim, max_seqs, max_tokens) < 1:
            _refuse("the sizes of a cache must be positive")
        self.torch = torch
        dtype = torch.bfloat16 if dtype is None else dtype
        per_page = (page_size, n_kv) if layout == "NHD" else (n_kv, page_size)
        k = torch.zeros((n_layers, num_pages) + per_page + (head_dim,), dtype=torch.uint8 if dtype.itemsize == 1 else dtype,
                        device=device).view(dtype)
        self.cache = MoeKvCache(k, torch.zeros_like(k.view(torch.uint8)).view(dtype), layout, k_scale, v_scale)
        self.device = k.device
        self.page_size, self.num_pages, self.max_seqs = page_size, num_pages, max_seqs
        self.max_pages = -(-max_tokens // page_size)
        self.max_tokens = max_tokens
        self.block_tables = torch.full((max_seqs, self.max_pages), -1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self.ops = LibmoeCacheOps() if ops is None else ops
        self._refs = [0] * num_pages                  # rows that hold a page
        self._free = list(range(num_pages))           # a heap: the lowest pages first
        self._rows = {}                               # open row -> its pages
        self._len = {}                                # open row -> its tokens
        self._free_rows = list(range(max_seqs))

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def pages_of(self, row: int) -> list[int]:
        """The pages of an open row, in order."""
        return list(self._pages(row))

    def length(self, row: int) -> int:
        self._pages(row)
        return self._len[row]

    def _pages(self, row):
        if row not in self._rows:
            _refuse(f"row {row} is not open")
        return self._rows[row]

    def _upload(self, tables, lens):
        """Block-table entries {(row, column): page} and lengths {row: tokens} to the device, without waiting."""
        torch = self.torch
        if not tables and not lens:
            return
        flat = [r * self.max_pages + c for r, c in tables] + list(tables.values()) + list(lens) + list(lens.values())
        host = torch.tensor(flat, dtype=torch.int64)
        if self.device.type == "cuda":
            host = host.pin_memory()
        dev = host.to(self.device, non_blocking=True)
        n, m = len(tables), len(lens)
        if n:
            self.block_tables.view(-1)[dev[:n]] = dev[n: 2 * n].to(torch.int32)
        if m:
            self.seq_lens[dev[2 * n: 2 * n + m]] = dev[2 * n + m:].to(torch.int32)

    def open(self) -> int:
        """A row for a new, empty sequence."""
        if not self._free_rows:
            _refuse(f"all {self.max_seqs} rows are open")
        row = heapq.heappop(self._free_rows)
        self._rows[row], self._len[row] = [], 0
        self._upload({}, {row: 0})
        return row

    def append(self, rows, counts):
        """Room for counts[i] new tokens of rows[i]: (positions int32, slots int64) of all of them, row after row,
        on the device; lengths and block tables there include them. Refused as a whole where the pages do not
        suffice."""
        torch = self.torch
        rows, counts = list(rows), list(counts)
        if len(rows) != len(counts) or len(set(rows)) != len(rows):
            _refuse("append: one count for each of some different rows")
        refs = {}   # changed reference counts, so that nothing is changed before all is known to fit
        need, plan = 0, []
        for row, n in zip(rows, counts):
            pages, have = self._pages(row), self._len[row]
            if n < 0 or have + n > self.max_tokens:
                _refuse(f"row {row}: {have} + {n} tokens, {self.max_tokens} at most")
            last = pages[-1] if n and have % self.page_size else None
            shared = last is not None and refs.get(last, self._refs[last]) > 1
            if shared:
                refs[last] = refs.get(last, self._refs[last]) - 1
            fresh = -(-(have + n) // self.page_size) - len(pages)
            need += fresh + shared
            plan.append((row, have, n, fresh, shared))
        if need > len(self._free):
            _refuse(f"append: {need} pages needed, {len(self._free)} free")
        src, dst, tables, lens, parts = [], [], {}, {}, []
        for row, have, n, fresh, shared in plan:
            pages = self._rows[row]
            if shared:
                page = self._take()
                self._refs[pages[-1]] -= 1
                src.append(pages[-1])
                dst.append(page)
                pages[-1] = page
                tables[row, len(pages) - 1] = page
            for _ in range(fresh):
                pages.append(self._take())
                tables[row, len(pages) - 1] = pages[-1]
            if n:
                self._len[row] = lens[row] = have + n
            t = torch.arange(have, have + n)
            first = have // self.page_size
            page = torch.tensor(pages[first:], dtype=torch.int64)[t // self.page_size - first] if n else t
            parts.append(torch.stack((t, page * self.page_size + t % self.page_size)))
        if src:
            self.ops.copy_pages(self.cache, src, dst)
        self._upload(tables, lens)
        host = torch.cat(parts, dim=1) if parts else torch.empty((2, 0), dtype=torch.int64)
        if self.device.type == "cuda":
            host = host.pin_memory()
        dev = host.to(self.device, non_blocking=True)
        return dev[0].to(torch.int32), dev[1].contiguous()

    def _take(self) -> int:
        page = heapq.heappop(self._free)
        self._refs[page] = 1
        return page

    def fork(self, row: int) -> int:
        """A new row with the same tokens; the pages are shared until one of the two writes its last one."""
        pages = self._pages(row)
        new = self.open()
        self._rows[new], self._len[new] = list(pages), self._len[row]
        for page in pages:
            self._refs[page] += 1
        self._upload({(new, c): page for c, page in enumerate(pages)}, {new: self._len[new]})
        return new

    def close(self, row: int) -> None:
        """Ends a sequence."""
        for page in self._pages(row):
            self._refs[page] -= 1
            if self._refs[page] == 0:
                heapq.heappush(self._free, page)
        del self._rows[row], self._len[row]
        heapq.heappush(self._free_rows, row)
        self._upload({}, {row: 0})

    def compact(self) -> int:
        """Moves the live pages to the front; returns how many moved. Pages from the live count on are free then."""
        live = self.num_pages - len(self._free)
        src = [p for p in range(live, self.num_pages) if self._refs[p]]
        if not src:
            return 0
        dst = [p for p in range(live) if not self._refs[p]]
        to = dict(zip(src, dst))
        self.ops.copy_pages(self.cache, src, dst, block_tables=self.block_tables)
        for pages in self._rows.values():
            pages[:] = [to.get(p, p) for p in pages]
        for a, b in to.items():
            self._refs[b], self._refs[a] = self._refs[a], 0
        self._free = list(range(live, self.num_pages))   # sorted: a heap
        return len(src)
