"""Definition of the pool's calls on plain lists: the block table, reference counts and which page holds a copy of which."""

from __future__ import annotations

import numpy as np

PAGE = 64


class Pool:
    def __init__(self, n_seqs, max_pages, n_pages, max_seq_len):
        self.table = np.full((n_seqs, max_pages), -1)
        self.n_pages, self.max_seq_len = n_pages, max_seq_len
        self.holds = np.arange(n_pages)                      # whose first contents a page holds
        self.flags = 0

    @property
    def refs(self):
        return np.bincount(self.table[self.table >= 0], minlength=self.n_pages)

    def reserve(self, pos, counts):
        """granted; NO_PAGES = 32, POS_RANGE = 2 in flags."""
        refs, B = self.refs, len(pos)
        ranges, granted = [], []
        for b, (p, n) in enumerate(zip(pos, counts)):
            n = max(n, 0)
            if p >= 0 and p + n > self.max_seq_len:
                self.flags |= 2
                p = -1
            granted.append(p)
            ranges.append(range(p // PAGE, (p + n - 1) // PAGE + 1) if p >= 0 and n > 0 else range(0))
        writers = {}
        for b in range(B):
            for lp in ranges[b]:
                e = self.table[b, lp]
                if e >= 0 and refs[e] > 1:
                    writers.setdefault(e, []).append((b, lp))
        free = [p for p in range(self.n_pages) if refs[p] == 0]
        plans, full = [], False
        for b in range(B):
            plan = []
            for lp in ranges[b]:
                e = self.table[b, lp]
                keeps = e >= 0 and (refs[e] <= 1 or (len(writers[e]) == refs[e] and writers[e][-1] == (b, lp)))
                if not keeps:
                    plan.append((lp, e))
            full |= len(plan) > len(free)
            if full:
                if granted[b] >= 0:
                    self.flags |= 32
                granted[b] = -1
                continue
            plans += [(b, lp, e, free.pop(0)) for lp, e in plan]
        for b, lp, e, page in plans:
            if e >= 0:
                self.holds[page] = self.holds[e]
            self.table[b, lp] = page
        return granted

    def fork(self, parents, lens):
        old, new = self.table.copy(), list(lens)
        for b, q in enumerate(parents):
            if q < -1 or q >= len(parents):
                self.flags |= 64
            if 0 <= q < len(parents) and q != b:
                n = -(-lens[q] // PAGE)
                self.table[b] = -1
                self.table[b, :n] = old[q, :n]
                new[b] = lens[q]
        return new

    def release(self, keep):
        for b, n in enumerate(keep):
            if n >= 0:
                self.table[b, -(-n // PAGE):] = -1

    def compact(self):
        refs = self.refs
        used = int((refs > 0).sum())
        holes = [p for p in range(used) if refs[p] == 0]
        movers = [p for p in range(used, self.n_pages) if refs[p] > 0]
        for src, dst in zip(movers, holes):
            self.holds[dst] = self.holds[src]
            self.table[self.table == src] = dst
        return used
