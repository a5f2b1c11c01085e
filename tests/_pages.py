"""The pages' bookkeeping on the host, one page at a time (include/csa.h)."""
import numpy as np


class Pages:
    """A table, lengths and counts as numpy int32; calls change them as the library's do and return what it writes.
    `refused` is set by a sequence that a call leaves as it is."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs = (np.array(x, dtype=np.int32) for x in (table, lens, refs))
        self.page, self.refused = page, False

    def count(self, tokens):
        return -(-int(tokens) // self.page)

    def length(self, b):
        return min(max(int(self.lens[b]), 0), self.table.shape[1] * self.page)

    def is_page(self, p):
        return 0 <= p < len(self.refs)

    def drop(self, refs, p):
        if self.is_page(p) and refs[p] > 0:
            refs[p] -= 1
        else:
            self.refused = True

    def resize(self, target, copies=True):
        n, P = len(self.lens), self.page
        free = [int(p) for p in np.flatnonzero(self.refs <= 0)]
        refs, lens = self.refs.copy(), self.lens.copy()
        pos0, src, dst = (np.full(n, -1, np.int32) for _ in range(3))
        taken = 0
        for b, t in enumerate(int(x) for x in target):
            L = self.length(b)
            lens[b] = L
            if t > self.table.shape[1] * P:
                self.refused = True
            elif t > L:
                old = int(self.table[b, L // P]) if L % P else -1
                if L % P and not self.is_page(old):
                    self.refused = True
                apart = L % P > 0 and self.is_page(old) and self.refs[old] > 1
                slots = ([L // P] if apart else []) + list(range(self.count(L), self.count(t)))
                first, taken = taken, taken + len(slots)
                if slots and taken > len(free) or apart and not copies:
                    self.refused = True
                    continue
                for i, j in enumerate(slots):
                    self.table[b, j] = free[first + i]
                    refs[free[first + i]] = 1
                if apart:
                    src[b], dst[b] = old, free[first]
                    self.drop(refs, old)
                pos0[b], lens[b] = L, t
            elif 0 <= t < L:
                for j in range(self.count(t), self.count(L)):
                    self.drop(refs, int(self.table[b, j]))
                    self.table[b, j] = -1
                lens[b] = t
        self.refs, self.lens = refs, lens
        return pos0, src, dst

    def fork(self, parent):
        n, P = len(self.lens), self.page
        free = [int(p) for p in np.flatnonzero(self.refs <= 0)]
        refs, lens, taken = self.refs.copy(), self.lens.copy(), 0
        src, dst = (np.full(n, -1, np.int32) for _ in range(2))
        for b, a in enumerate(int(x) for x in parent):
            if a < 0:
                continue
            if a >= n or self.lens[b] > 0:
                self.refused = True
                continue
            L = self.length(a)
            if L == 0:
                continue
            if L % P:
                taken += 1
                if taken > len(free):
                    self.refused = True
                    continue
                last = int(self.table[a, L // P])
                self.table[b, L // P] = free[taken - 1]
                refs[free[taken - 1]] = 1
                if self.is_page(last):
                    src[b], dst[b] = last, free[taken - 1]
                else:
                    self.refused = True
            for j in range(L // P):
                p = int(self.table[a, j])
                self.table[b, j] = p
                if self.is_page(p):
                    refs[p] += 1
                else:
                    self.refused = True
            lens[b] = L
        self.refs, self.lens = refs, lens
        return src, dst

    def compact(self):
        """(src, dst, used); the table and the counts are renumbered."""
        n = len(self.refs)
        used = self.refs > 0
        U = int(used.sum())
        src, dst = (np.full(n // 2, -1, np.int32) for _ in range(2))
        late, holes = [p for p in range(U, n) if used[p]], [p for p in range(U) if not used[p]]
        assert len(late) == len(holes)
        src[:len(late)], dst[:len(late)] = late, holes
        to = dict(zip(late, holes))
        refs = np.where(used, self.refs, 0).astype(np.int32)
        for a, b in to.items():
            refs[a], refs[b] = 0, self.refs[a]
        for b in range(len(self.lens)):
            for j in range(self.count(self.length(b))):
                p = int(self.table[b, j])
                if not self.is_page(p):
                    self.refused = True
                self.table[b, j] = to.get(p, p)
        self.refs = refs
        return src, dst, U

    def check(self):
        """Every page's count is the number of entries that hold it."""
        n = np.zeros(len(self.refs), np.int64)
        for b in range(len(self.lens)):
            np.add.at(n, self.table[b, :self.count(self.lens[b])], 1)
        assert (n == self.refs).all()
