"""Oracle for the page bookkeeping: a pool kept in plain Python.

State: ``table`` [rows][width], ``held`` [rows] leading entries that name
pages, ``ctx`` [rows] tokens, ``refs`` [pages] entries naming each page.

Test infrastructure only.
"""

from __future__ import annotations

from typing import List, Sequence, Tuple


class Pool:
    def __init__(self, table, held, ctx, refs, page_size: int = 16):
        self.table = [[int(x) for x in row] for row in table]
        self.held = [int(x) for x in held]
        self.ctx = [int(x) for x in ctx]
        self.refs = [int(x) for x in refs]
        self.page = page_size

    def pages_for(self, tokens: int) -> int:
        return -(-tokens // self.page)

    def check(self) -> None:
        """Every reference is an entry: the invariant all operations keep."""
        count = [0] * len(self.refs)
        for row, n in zip(self.table, self.held):
            for page in row[:n]:
                count[page] += 1
        assert count == self.refs, (count, self.refs)

    def release(self, keep: Sequence[int]) -> None:
        for b, tokens in enumerate(keep):
            n = min(self.pages_for(int(tokens)), self.held[b])
            for lp in range(n, self.held[b]):
                self.refs[self.table[b][lp]] -= 1
                self.table[b][lp] = -1
            self.held[b] = n

    def fork(self, parents: Sequence[int], children: Sequence[int]) -> None:
        for parent, child in zip(parents, children):
            n = self.pages_for(self.ctx[parent])
            for lp in range(n):
                self.table[child][lp] = self.table[parent][lp]
                self.refs[self.table[parent][lp]] += 1
            self.held[child], self.ctx[child] = n, self.ctx[parent]

    def reserve(self, new: Sequence[int]) -> List[Tuple[int, int]]:
        """Returns the pages to copy as (old, new); raises MemoryError, with
        nothing changed, when the pool is too small."""
        ranges = []
        for b, tokens in enumerate(new):
            grows = int(tokens) > self.ctx[b]
            ranges.append((self.ctx[b] // self.page, self.pages_for(int(tokens))) if grows else (0, 0))
        writers = {}  # shared page -> rows of this call that write to it
        for b, (first, need) in enumerate(ranges):
            for lp in range(first, min(self.held[b], need)):
                if self.refs[self.table[b][lp]] > 1:
                    writers.setdefault(self.table[b][lp], []).append(b)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        taken, copies, changes = 0, [], []
        for b, (first, need) in enumerate(ranges):
            for lp in range(first, need):
                old = None
                if lp < self.held[b]:
                    old = self.table[b][lp]
                    rows = writers.get(old)
                    if rows is None or (len(rows) == self.refs[old] and rows[0] == b):
                        continue
                if taken == len(free):
                    raise MemoryError("pool")
                changes.append((b, lp, old, free[taken]))
                if old is not None and lp == first and self.ctx[b] % self.page:
                    copies.append((old, free[taken]))
                taken += 1
        for b, lp, old, page in changes:
            if old is not None:
                self.refs[old] -= 1
            self.refs[page] = 1
            self.table[b][lp] = page
            self.held[b] = max(self.held[b], lp + 1)
        return copies

    def compact(self) -> Tuple[List[Tuple[int, int]], int]:
        """Returns (moves as (old, new), pages in use)."""
        live = sum(r > 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= live]
        dst = [p for p, r in enumerate(self.refs) if r == 0 and p < live]
        move = dict(zip(src, dst))
        for row, n in zip(self.table, self.held):
            row[:n] = [move.get(p, p) for p in row[:n]]
        for a, z in move.items():
            self.refs[z], self.refs[a] = self.refs[a], 0
        return list(zip(src, dst)), live


def copy_pages(pool, pairs):
    """Pages ``pairs`` (source, destination) of a pool [layers, pages, ...]."""
    out = pool.copy()
    for a, z in pairs:
        out[:, z] = pool[:, a]
    return out
