"""A paged key-value cache: which pages each sequence owns.

The keys and values of all layers live in two pools [layers, pages, kv_heads,
page_size, head_dim]; a page is the same index in every layer.  This class does
the bookkeeping on the host (a free list, a count of owners per page, each
sequence's list of pages) and moves data with kv_copy_pages only, on the
current stream.  Forks share pages: a sequence gets its own copy of a shared
page when it first writes to it.
"""
from __future__ import annotations

import heapq
from typing import NamedTuple, Sequence

import torch

from . import _lib

PAGE_SIZES = tuple(1 << i for i in range(4, 11))


class CacheFull(RuntimeError):
    """Not enough free pages; the cache is as it was before the call."""


class Batch(NamedTuple):
    """One step's device arrays, as kv_append and the attention calls take them.
    (New ones each time, as wide as the step's longest sequence: a captured graph
    has its own and copies these into them.)"""
    table: torch.Tensor      # int32 [seqs, width]; -1 where a sequence owns no page
    lens: torch.Tensor       # int32 [seqs], the new tokens included
    starts: torch.Tensor     # int32 [seqs + 1]
    tokens: int
    max_len: int


class _Sequence:
    __slots__ = ("pages", "length")

    def __init__(self, pages, length):
        self.pages, self.length = pages, length


class KVCache:
    def __init__(self, layers: int, pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                 dtype: torch.dtype = torch.float16, device="cuda"):
        if min(layers, pages, kv_heads, head_dim, page_size) <= 0:
            raise ValueError("layers, pages, kv_heads, head_dim and page_size must be positive")
        if layers > 4096 or pages > 1 << 24:
            raise ValueError("at most 4096 layers and 2^24 pages")
        # What the calls on these pools would refuse later, with pages handed
        # out already.  (Pools on the host serve the bookkeeping alone.)
        if torch.device(device).type != "cpu":
            if dtype not in _lib._DTYPES:
                raise TypeError(f"the pools must be float16 or bfloat16, not {dtype}")
            if _lib.slim_attention_workspace_bytes(1, 1, kv_heads, kv_heads, head_dim) == 0:
                raise ValueError(f"no attention with {kv_heads} key heads of size {head_dim}")
            if page_size not in PAGE_SIZES:
                raise ValueError(f"page_size must be one of {PAGE_SIZES}, not {page_size}")
        self.page_size = page_size
        self.k = torch.empty((layers, pages, kv_heads, page_size, head_dim), dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        self._owners = [0] * pages
        self._free = list(range(pages))      # a heap: the lowest free page goes out first
        self._seqs: dict[int, _Sequence] = {}
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self._seqs[seq].length

    def pages(self, seq: int) -> list[int]:
        """The pages of a sequence in order; -1 where drop() gave one back."""
        return list(self._seqs[seq].pages)

    def add(self) -> int:
        """A new, empty sequence."""
        return self._put(_Sequence([], 0))

    def _put(self, s: _Sequence) -> int:
        seq, self._next = self._next, self._next + 1
        self._seqs[seq] = s
        return seq

    def fork(self, seq: int) -> int:
        """A new sequence with the tokens of `seq`; it shares the pages."""
        s = self._seqs[seq]
        for p in s.pages:
            if p >= 0:
                self._owners[p] += 1
        return self._put(_Sequence(list(s.pages), s.length))

    def free(self, seq: int) -> None:
        """Give up a sequence; pages that nobody else owns become free."""
        s = self._seqs.pop(seq)
        for p in s.pages:
            self._release(p)

    def _release(self, p: int) -> None:
        if p < 0:
            return
        self._owners[p] -= 1
        if self._owners[p] == 0:
            heapq.heappush(self._free, p)

    def drop(self, seq: int, window: int, sinks: int = 0) -> int:
        """Give back the pages that no later token of `seq` sees under a
        sliding window with `sinks` first tokens; returns how many."""
        if window <= 0 or sinks < 0:
            raise ValueError("drop needs window > 0 and sinks >= 0")
        s, size = self._seqs[seq], self.page_size
        # The next token, at position length, sees length - window + 1 and
        # later, so a page that is still being filled stays.
        end, n = min(max(0, s.length - window + 1) // size, len(s.pages)), 0
        for i in range(-(-sinks // size), end):
            if s.pages[i] >= 0:
                self._release(s.pages[i])
                s.pages[i] = -1
                n += 1
        return n

    def extend(self, seqs: Sequence[int], counts: Sequence[int] | None = None) -> Batch:
        """Make room for counts[i] new tokens of sequence seqs[i] (one each if
        None) and return the step's batch; raises CacheFull if the free pages
        do not suffice.  After any error the cache is as it was."""
        seqs = list(seqs)
        counts = [1] * len(seqs) if counts is None else list(counts)
        if len(counts) != len(seqs) or len(set(seqs)) != len(seqs) or any(c < 0 for c in counts):
            raise ValueError("extend needs different sequences and a count >= 0 for each")
        size, need = self.page_size, 0
        # Owners that remain for a shared page as the sequences of this step take their own copies, in order.
        left: dict[int, int] = {}
        copies = []
        for q, c in zip(seqs, counts):
            s = self._seqs[q]
            need += max(0, -(-(s.length + c) // size) - len(s.pages))
            if c and s.length % size:
                p = s.pages[-1]
                n = left.get(p, self._owners[p])
                if n > 1:
                    left[p] = n - 1
                    copies.append(q)
                    need += 1
        if need > len(self._free):
            raise CacheFull(f"{need} pages needed, {len(self._free)} free")
        before = [(s, len(s.pages), s.length) for s in (self._seqs[q] for q in seqs)]
        src = [self._seqs[q].pages[-1] for q in copies]
        dst = [self._take() for _ in copies]
        try:
            self._move(src, dst)
            for q, p in zip(copies, dst):
                self._seqs[q].pages[-1] = p
            for q, c in zip(seqs, counts):
                s = self._seqs[q]
                s.length += c
                while len(s.pages) * size < s.length:
                    s.pages.append(self._take())
            batch = self.batch(seqs, counts)
        except BaseException:
            for s, n, length in before:
                for p in s.pages[n:]:
                    self._release(p)
                del s.pages[n:]
                s.length = length
            for q, p in zip(copies, src):
                self._seqs[q].pages[-1] = p
            for p in dst:
                self._release(p)
            raise
        for p in src:
            self._release(p)
        return batch

    def _take(self) -> int:
        p = heapq.heappop(self._free)
        self._owners[p] = 1
        return p

    def _move(self, src: list[int], dst: list[int]) -> None:
        if src:
            ids = torch.tensor([src, dst], dtype=torch.int32).to(self.k.device)
            _lib.slim_kv_copy_pages(self.k, self.v, ids[0], ids[1])

    def batch(self, seqs: Sequence[int], counts: Sequence[int] | None = None) -> Batch:
        """The device arrays of a step whose last counts[i] tokens of seqs[i] are the new ones."""
        seqs = list(seqs)
        counts = [1] * len(seqs) if counts is None else list(counts)
        rows = [self._seqs[q] for q in seqs]
        width = max([len(s.pages) for s in rows] + [1])
        flat = [p for s in rows for p in s.pages + [-1] * (width - len(s.pages))]
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + c)
        n, lens = len(rows), [s.length for s in rows]
        ints = torch.tensor(flat + lens + starts, dtype=torch.int32).to(self.k.device)     # one copy
        return Batch(ints[:n * width].view(n, width), ints[n * width:n * width + n], ints[n * width + n:], starts[-1],
                     max(lens, default=0))

    def compact(self) -> int:
        """Move the pages in use to the lowest indices, so that all free ones
        lie behind them; returns how many moved.  Batches made before are
        stale."""
        live = sum(1 for n in self._owners if n)
        src = [p for p in range(live, len(self._owners)) if self._owners[p]]
        dst = [p for p in range(live) if not self._owners[p]]
        self._move(src, dst)
        to = dict(zip(src, dst))
        for p, q in to.items():
            self._owners[q], self._owners[p] = self._owners[p], 0
        for s in self._seqs.values():
            s.pages = [to.get(p, p) for p in s.pages]
        self._free = list(range(live, len(self._owners)))
        return len(src)
