"""Host-side bookkeeping of a paged cache: which pages are free, which sequences share which.

No tensor of the cache is touched here: methods that need pages copied return the page numbers
for attn_cache_copy.  A sequence is the list of its pages, in order, as this class gave them
out; page numbers go into the int32 tables of attn_cache_append and attn_decode_paged."""
from __future__ import annotations

import heapq

import torch


class CacheFull(RuntimeError):
    """The cache has fewer free pages than were asked for; nothing was changed."""


class CachePages:
    def __init__(self, pages: int, page: int):
        """`pages` pages of `page` tokens each, all free."""
        if pages <= 0 or page <= 0:
            raise ValueError("gbattn: pages and page must be positive")
        self.pages, self.page = int(pages), int(page)
        self._users = [0] * self.pages
        self._free = list(range(self.pages))  # a heap: the lowest free page is given out first

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def users(self, page: int) -> int:
        """How many sequences hold a page."""
        return self._users[page]

    def _take(self, n: int) -> list[int]:
        if n > len(self._free):
            raise CacheFull(f"gbattn: {n} pages asked for, {len(self._free)} free")
        got = [heapq.heappop(self._free) for _ in range(n)]
        for p in got:
            self._users[p] = 1
        return got

    def _check(self, sequence) -> None:
        for p in sequence:
            if not 0 <= p < self.pages or self._users[p] <= 0:
                raise ValueError(f"gbattn: page {p} is not in use")

    def _need(self, length: int) -> int:
        if length < 0:
            raise ValueError("gbattn: a length must not be negative")
        return -(-length // self.page)

    def new(self, length: int = 0) -> list[int]:
        """A sequence with room for `length` tokens."""
        return self._take(self._need(length))

    def grow(self, sequence: list[int], length: int, new_length: int) -> tuple[list[int], list[int]]:
        """Make room in `sequence` (changed in place) of `length` tokens for new_length tokens, and make the
        pages that tokens length .. new_length - 1 go to its own: a last page that is partly filled and
        shared is replaced.  Returns (src, dst), the pages to copy before tokens are appended."""
        self._check(sequence)
        if new_length < length or self._need(length) > len(sequence):
            raise ValueError("gbattn: grow needs length <= new_length and a sequence that holds length tokens")
        first, need = length // self.page, self._need(new_length)
        shared = [i for i in range(first, min(need, len(sequence))) if self._users[sequence[i]] > 1]
        fresh = self._take(len(shared) + max(0, need - len(sequence)))
        src, dst = [], []
        for i in shared:
            old, mine = sequence[i], fresh.pop(0)
            if i * self.page < length:  # it holds tokens
                src.append(old)
                dst.append(mine)
            self._users[old] -= 1
            sequence[i] = mine
        sequence.extend(fresh)
        return src, dst

    def fork(self, sequence: list[int], length: int) -> tuple[list[int], list[int], list[int]]:
        """A second sequence with the first `length` tokens of `sequence`: full pages are shared, a partly
        filled last one is copied.  Returns (its pages, src, dst)."""
        self._check(sequence)
        need, full = self._need(length), length // self.page
        if need > len(sequence):
            raise ValueError("gbattn: the sequence holds fewer tokens")
        last = self._take(need - full)
        for p in sequence[:full]:
            self._users[p] += 1
        return sequence[:full] + last, sequence[full:need], list(last)

    def free(self, sequence: list[int]) -> None:
        """Give up a sequence (emptied in place); pages that nobody else holds become free."""
        self._check(sequence)
        if len(set(sequence)) != len(sequence):
            raise ValueError("gbattn: a page occurs twice in a sequence")
        for p in sequence:
            self._users[p] -= 1
            if self._users[p] == 0:
                heapq.heappush(self._free, p)
        sequence.clear()

    def compact(self, sequences: list[list[int]]) -> tuple[list[int], list[int]]:
        """Move the pages in use to the lowest numbers.  `sequences`: all that hold pages (changed in
        place).  Returns (src, dst), the pages to copy: each source lies above every destination."""
        held = [0] * self.pages
        for s in sequences:
            self._check(s)
            for p in s:
                held[p] += 1
        if held != self._users:
            raise ValueError("gbattn: compact needs every sequence that holds pages, once")
        used = self.pages - len(self._free)
        src = [p for p in range(used, self.pages) if self._users[p]]
        dst = [p for p in range(used) if not self._users[p]]
        to = dict(zip(src, dst))
        for s in sequences:
            s[:] = [to.get(p, p) for p in s]
        for a, b in to.items():
            self._users[b], self._users[a] = self._users[a], 0
        self._free = list(range(used, self.pages))
        return src, dst

    def table(self, sequences: list[list[int]], width: int | None = None) -> torch.Tensor:
        """The int32 page table [len(sequences), width] on the host, -1 behind a sequence's last page."""
        longest = max((len(s) for s in sequences), default=0)
        width = max(1, longest) if width is None else width
        if longest > width:
            raise ValueError("gbattn: a sequence has more pages than the table's width")
        return torch.tensor([s + [-1] * (width - len(s)) for s in sequences], dtype=torch.int32).reshape(-1, width)
