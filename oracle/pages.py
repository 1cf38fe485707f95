"""CPU oracle of the paged cache -- TEST INFRASTRUCTURE ONLY.

The operators of include/pagecache.h, one request at a time on 64-bit numpy
arrays, written for a reader to check by eye. It shares nothing with the CUDA
library. A page is free when no row names it, so the oracle keeps references
and derives the free pages from them.
"""

from __future__ import annotations

import numpy as np

NONE = -1
ALL = 0xFFFFFFFF
OK, INVALID, SHORT = 0, 1, 2


def pack_free(refs) -> np.ndarray:
    """The free pages as 32-bit words, bit p % 32 of word p // 32."""
    refs = np.asarray(refs)
    words = np.zeros((refs.size + 31) // 32, dtype=np.uint32)
    for p in np.flatnonzero(refs == 0):
        words[p // 32] |= np.uint32(1) << np.uint32(p % 32)
    return words


class Cache:
    def __init__(self, n_seqs: int, columns: int, n_pages: int, page_tokens: int):
        self.T = page_tokens
        self.table = np.full((n_seqs, columns), NONE, dtype=np.int64)
        self.length = np.zeros(n_seqs, dtype=np.int64)
        self.refs = np.zeros(n_pages, dtype=np.int64)

    def copy(self) -> "Cache":
        c = Cache(self.table.shape[0], self.table.shape[1], self.refs.size, self.T)
        c.table, c.length, c.refs = self.table.copy(), self.length.copy(), self.refs.copy()
        return c

    def pages(self, tokens: int) -> int:
        return -(-int(tokens) // self.T)

    def lowest_free(self) -> int:
        free = np.flatnonzero(self.refs == 0)
        return int(free[0]) if free.size else -1

    # Each call returns (status, counters, ...) and changes the cache.
    def free(self, req):
        seen, status, released, invalid = set(), [], 0, 0
        for seq, keep in np.asarray(req, dtype=np.int64).reshape(-1, 2).tolist():
            if not 0 <= seq < self.length.size or seq in seen:
                status.append(INVALID)
                invalid += 1
                continue
            seen.add(seq)
            status.append(OK)
            if keep >= self.length[seq]:
                continue
            for c in range(self.pages(keep), self.pages(self.length[seq])):
                page = self.table[seq, c]
                self.refs[page] -= 1
                if self.refs[page] == 0:
                    released += 1
                self.table[seq, c] = NONE
            self.length[seq] = keep
        return status, [released, invalid, 0, 0]

    def fork(self, req):
        before = self.length.copy()
        seen, status, taken, invalid = set(), [], 0, 0
        n = before.size
        for parent, child, tokens, _ in np.asarray(req, dtype=np.int64).reshape(-1, 4).tolist():
            first = 0 <= child < n and child not in seen
            if first:
                seen.add(child)
            if not (first and 0 <= parent < n and parent != child and before[child] == 0
                    and 0 <= tokens <= before[parent]):
                status.append(INVALID)
                invalid += 1
                continue
            status.append(OK)
            for c in range(self.pages(tokens)):
                page = self.table[parent, c]
                self.table[child, c] = page
                self.refs[page] += 1
                taken += 1
            self.length[child] = tokens
        return status, [taken, invalid, 0, 0]

    def extend(self, req):
        """Returns (status, counters, moves)."""
        req = np.asarray(req, dtype=np.int64).reshape(-1, 2).tolist()
        was = self.copy()
        free = np.flatnonzero(self.refs == 0).tolist()  # the lowest first
        seen, status, moves, need, invalid = set(), [], [], 0, 0

        def take():
            nonlocal need
            need += 1
            if need > len(free):
                return None
            self.refs[free[need - 1]] = 1
            return free[need - 1]

        for seq, tokens in req:
            first = 0 <= seq < self.length.size and seq not in seen
            if first:
                seen.add(seq)
            now = int(self.length[seq]) + tokens if first else 0
            if not first or tokens < 0 or now > self.table.shape[1] * self.T or now >= 2**32:
                status.append(INVALID)
                invalid += 1
                continue
            status.append(OK)
            length = int(self.length[seq])
            last = self.pages(length) - 1
            if tokens > 0 and length % self.T != 0 and self.refs[self.table[seq, last]] > 1:
                shared = int(self.table[seq, last])
                page = take()
                self.refs[shared] -= 1
                if page is not None:
                    self.table[seq, last] = page
                    moves.append([shared, page, length % self.T, 0])
            for c in range(self.pages(length), self.pages(now)):
                page = take()
                if page is not None:
                    self.table[seq, c] = page
            self.length[seq] = now
        if need > len(free):  # all or nothing
            self.table, self.length, self.refs = was.table, was.length, was.refs
            status = [SHORT if s == OK else s for s in status]
            return status, [need, invalid, len(status) - invalid, 0], []
        return status, [need, invalid, 0, 0], moves

    def compact(self, cap: int):
        """Returns (counters, moves)."""
        moves = []
        possible = 0
        refs = self.refs.copy()
        live = int((refs > 0).sum())
        lo, hi = 0, refs.size - 1
        while True:
            while lo < refs.size and refs[lo] > 0:
                lo += 1
            while hi >= 0 and refs[hi] == 0:
                hi -= 1
            if lo >= hi or lo >= live:
                break
            if possible < cap:
                moves.append([hi, lo, ALL, 0])
                self.refs[lo], self.refs[hi] = self.refs[hi], 0
                self.table[self.table == hi] = lo
            refs[lo], refs[hi] = refs[hi], 0
            possible += 1
        return [possible, 0, possible - len(moves), 0], moves


def copy(moves, src: np.ndarray, dst: np.ndarray, token_dim: int | None) -> None:
    """The moves' bytes between pools [planes, pages, ...] (in place)."""
    for s, d, tokens, _ in np.asarray(moves, dtype=np.int64).reshape(-1, 4).tolist():
        if s >= src.shape[1] or d >= dst.shape[1]:
            continue
        if token_dim is None:
            if tokens:
                dst[:, d] = src[:, s]
            continue
        for t in range(min(tokens, src.shape[token_dim])):
            at = (slice(None),) * (token_dim - 2) + (t,)
            dst[(slice(None), d) + at] = src[(slice(None), s) + at]


def check(c: Cache) -> None:
    """What holds of every cache: rows hold pages up to their length and none past it, a row
    names a page once, and references count the rows that name a page."""
    count = np.zeros(c.refs.size, dtype=np.int64)
    for s in range(c.length.size):
        n = c.pages(c.length[s])
        row = c.table[s]
        assert (row[:n] >= 0).all() and (row[:n] < c.refs.size).all() and (row[n:] == NONE).all()
        assert len(set(row[:n].tolist())) == n
        count[row[:n]] += 1
    assert (count == c.refs).all()
