"""Host side of the paged key/value cache: which sequence holds which pages.

:class:`PagePool` hands out the pages of a cache whose tensors the caller owns
(layout: include/attn_core.h), keeps each sequence's page list and length, and
says which pages have to be copied: a fork shares its parent's pages until one
of the two writes into a shared page, and compaction moves pages to the free
places of lowest number.  The copies are lists of (from, to) for
``page_copy``, to be made on the stream of the calls that follow, before them.

Pure Python on the host, no GPU: a page's number is the same in every layer's
planes, so one pool serves a whole model.
"""
from __future__ import annotations

import heapq

import numpy as np

__all__ = ["OutOfPages", "PagePool"]


class OutOfPages(RuntimeError):
    """The cache has fewer free pages than were asked for; nothing was changed."""


class PagePool:
    def __init__(self, n_pages: int, page_size: int):
        if n_pages < 1 or page_size < 1:
            raise ValueError("n_pages and page_size must be positive")
        self.n_pages, self.page_size = int(n_pages), int(page_size)
        self._free = list(range(self.n_pages))      # a heap: the lowest number first
        self._users = [0] * self.n_pages            # sequences that hold each page
        self._pages: dict[int, list[int]] = {}
        self._length: dict[int, int] = {}
        self._next = 0

    # ------------------------------------------------------------ queries ---
    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self._length[seq]

    def pages(self, seq: int) -> list[int]:
        return list(self._pages[seq])

    def tables(self, seqs, max_pages: int):
        """(page_table int32 [n, max_pages], kv_lens int32 [n]) of these
        sequences, for the device tables; unused entries are -1."""
        table = np.full((len(seqs), int(max_pages)), -1, dtype=np.int32)
        for i, s in enumerate(seqs):
            p = self._pages[s]
            if len(p) > max_pages:
                raise ValueError(f"sequence {s} has {len(p)} pages, more than the table's {max_pages}")
            table[i, :len(p)] = p
        return table, np.array([self._length[s] for s in seqs], dtype=np.int32)

    def groups(self, seqs):
        """(group_starts int32 [n_groups + 1], prefix_pages int32 [n_groups]) of
        neighbours among these sequences that share their first pages, for
        ``paged_prefix_fwd``.  Of nested choices (a system prompt that all share, a
        document that some do) the batch takes those that save the most page visits,
        (sequences - 1) * pages summed over the groups.  What this finds holds until a
        fork, a copy that ``extend`` asks for, ``truncate``, ``shrink`` or another list of
        sequences; tokens that are added in between change nothing (64 forks take
        1.2 ms of the host, so it is not asked at each step)."""
        n = len(seqs)
        if n == 0:
            raise ValueError("no sequences")
        # best[j]: the most that the first j sequences save; min_common[i]: what the
        # sequences i .. j - 1 have in common
        best, start_of = np.zeros(n + 1, dtype=np.int64), np.zeros(n + 1, dtype=np.int64)
        min_common, low, shared_of = np.zeros(n, dtype=np.int64), 0, np.zeros(n + 1, dtype=np.int64)
        members = np.arange(n, 0, -1, dtype=np.int64)
        for j in range(1, n + 1):
            if j > 1:
                pages = self._common(seqs[j - 2], seqs[j - 1])
                if pages == 0:
                    low = j - 1                 # no group reaches across
                else:
                    np.minimum(min_common[low:j - 1], pages, out=min_common[low:j - 1])
            min_common[j - 1] = np.iinfo(np.int64).max // (2 * n)
            total = best[low:j] + min_common[low:j] * (members[n - j + low:n] - 1)
            i = low + int(np.argmax(total))
            best[j], start_of[j] = total[i - low], i
            shared_of[j] = min_common[i] if i < j - 1 else 0
        starts, shared, j = [n], [], n
        while j > 0:
            shared.append(shared_of[j])
            j = int(start_of[j])
            starts.append(j)
        return np.array(starts[::-1], dtype=np.int32), np.array(shared[::-1], dtype=np.int32)

    def _common(self, a: int, b: int) -> int:
        """First pages that two sequences have in common."""
        x, y = self._pages[a], self._pages[b]
        n = min(len(x), len(y))
        if x[:n] == y[:n]:
            return n
        lo, hi = 0, n                           # shared pages come first, so halving finds the border
        while lo < hi:
            mid = (lo + hi) // 2
            if x[mid] == y[mid]:
                lo = mid + 1
            else:
                hi = mid
        return lo

    # ------------------------------------------------------------ changes ---
    def _take(self) -> int:
        page = heapq.heappop(self._free)
        self._users[page] = 1
        return page

    def _drop(self, page: int) -> None:
        self._users[page] -= 1
        if self._users[page] == 0:
            heapq.heappush(self._free, page)

    def add(self) -> int:
        """A new, empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._pages[seq], self._length[seq] = [], 0
        return seq

    def fork(self, seq: int) -> int:
        """A new sequence with the same keys and values, sharing every page."""
        pages, length = list(self._pages[seq]), self._length[seq]
        new = self.add()
        self._pages[new], self._length[new] = pages, length
        for page in pages:
            self._users[page] += 1
        return new

    def extend(self, seq: int, n: int) -> list[tuple[int, int]]:
        """Room for n more tokens of a sequence.  Returns the copies to make
        before they are written: the last page, where it is partly filled and
        another sequence holds it too."""
        if n < 0:
            raise ValueError("n must not be negative")
        pages, length = self._pages[seq], self._length[seq]
        need = -(-(length + n) // self.page_size) - len(pages)
        shared = n > 0 and length % self.page_size != 0 and self._users[pages[-1]] > 1
        if need + shared > len(self._free):
            raise OutOfPages(f"{need + shared} pages wanted, {len(self._free)} free")
        copies = []
        if shared:
            old, pages[-1] = pages[-1], self._take()
            copies.append((old, pages[-1]))
            self._drop(old)
        pages.extend(self._take() for _ in range(need))
        self._length[seq] = length + n
        return copies

    def truncate(self, seq: int, length: int) -> None:
        """Forget a sequence's tokens from position ``length`` on."""
        if not 0 <= length <= self._length[seq]:
            raise ValueError(f"length must be in 0 .. {self._length[seq]}")
        pages, keep = self._pages[seq], -(-length // self.page_size)
        while len(pages) > keep:
            self._drop(pages.pop())
        self._length[seq] = length

    def shrink(self, seqs, lengths, max_pages: int) -> np.ndarray:
        """These sequences keep ``lengths[i]`` keys each (``paged_evict``, one call for
        all of them).  Returns its out_table int32 [n, max_pages]: the sequence's own
        pages, and fresh ones in the places of those that another sequence holds too.
        What is not needed any more is free afterwards; the eviction has to be queued
        before anything that writes there."""
        if len(set(seqs)) != len(seqs) or len(seqs) != len(lengths):
            raise ValueError("each sequence is named once, with its length")
        take = 0
        for s, n in zip(seqs, lengths):
            if not 0 <= n <= self._length[s]:
                raise ValueError(f"length of sequence {s} must be in 0 .. {self._length[s]}")
            need = -(-n // self.page_size)
            if need > max_pages:
                raise ValueError(f"sequence {s} keeps {need} pages, more than the table's {max_pages}")
            take += sum(self._users[p] > 1 for p in self._pages[s][:need])
        if take > len(self._free):
            raise OutOfPages(f"{take} pages wanted, {len(self._free)} free")
        table = np.full((len(seqs), int(max_pages)), -1, dtype=np.int32)
        gone = []
        # by the holders before the call: a page that two of the sequences leave is read by both
        shared = {p for s in seqs for p in self._pages[s] if self._users[p] > 1}
        for i, (s, n) in enumerate(zip(seqs, lengths)):
            old, need = self._pages[s], -(-n // self.page_size)
            new = [self._take() if p in shared else p for p in old[:need]]
            stays = set(new)
            gone += [p for p in old if p not in stays]
            table[i, :need] = new
            self._pages[s], self._length[s] = new, n
        for p in gone:
            self._drop(p)
        return table

    def free(self, seq: int) -> None:
        """The sequence and its hold on its pages are gone."""
        for page in self._pages.pop(seq):
            self._drop(page)
        del self._length[seq]

    def compact(self) -> list[tuple[int, int]]:
        """Moves pages so that those in use have the lowest numbers.  Returns
        the copies; no target is another copy's source."""
        used = self.n_pages - len(self._free)
        holes = sorted(p for p in self._free if p < used)
        movers = [p for p in range(used, self.n_pages) if self._users[p]]
        to = dict(zip(movers, holes))
        for src, dst in to.items():
            self._users[dst], self._users[src] = self._users[src], 0
        for pages in self._pages.values():
            pages[:] = [to.get(p, p) for p in pages]
        self._free = list(range(used, self.n_pages))
        return list(to.items())
