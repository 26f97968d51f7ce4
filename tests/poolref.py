"""Plain reference of the page pool, in loops: fork, reserve, free and compact as
pq.h states them, with the codes of every layer."""
from __future__ import annotations

import numpy as np


class Pool:
    """A host copy of a pool and its layers' caches."""

    def __init__(self, n_seq, table_ld, n_pages, page, layers, seed):
        rng = np.random.default_rng(seed)
        self.n_seq, self.table_ld, self.n_pages, self.page, self.layers = n_seq, table_ld, n_pages, page, layers
        self.refs = np.zeros(n_pages, np.int32)
        self.table = np.full((n_seq, table_ld), -1, np.int32)
        self.len = np.zeros(n_seq, np.int32)
        self.codes = [[rng.integers(-127, 128, (n_pages, n_kv, page, d)).astype(np.int8) for _ in range(2)] for n_kv, d in layers]
        self.scales = [[rng.random((n_pages, n_kv)).astype(np.float32) for _ in range(2)] for n_kv, _ in layers]

    def fill(self, lens, seed, room=0):
        """Sequences of these lengths in scattered pages, with room for some more tokens."""
        order, at = np.random.default_rng(seed).permutation(self.n_pages), 0
        for s, n in enumerate(lens):
            m = min(-(-(n + room) // self.page), self.table_ld) if n else 0
            self.table[s, :m] = order[at:at + m]
            self.refs[order[at:at + m]] = 1
            at += m
            self.len[s] = n
        assert at <= self.n_pages

    def names(self, p):
        return 0 <= p < self.n_pages

    def check(self):
        """refs is the number of entries that name a page."""
        named = self.table[(self.table >= 0) & (self.table < self.n_pages)]
        assert np.array_equal(np.bincount(named, minlength=self.n_pages), self.refs)

    def fork(self, frm, to, tokens=None):
        table, lens = self.table.copy(), self.len.copy()
        seen = set()
        for i, (f, t) in enumerate(zip(frm, to)):
            if not (0 <= f < self.n_seq and 0 <= t < self.n_seq) or t in seen:
                continue
            seen.add(t)
            m = max(int(lens[f]), 0)
            if tokens is not None:
                m = min(m, max(int(tokens[i]), 0))
            row = np.full(self.table_ld, -1, np.int32)
            for j in range(min(-(-m // self.page), self.table_ld)):
                if self.names(table[f, j]):
                    row[j] = table[f, j]
                    self.refs[row[j]] += 1
            for p in table[t]:
                if self.names(p):
                    self.refs[p] -= 1
            self.table[t], self.len[t] = row, m

    def free(self, seq=None, begin=None, end=None, n=None):
        seq = list(range(n if n is not None else self.n_seq)) if seq is None else seq
        seen = set()
        for i, s in enumerate(seq):
            if not 0 <= s < self.n_seq or s in seen:
                continue
            seen.add(s)
            length = max(int(self.len[s]), 0)
            b = max(int(begin[i]), 0) if begin is not None else 0
            e = int(end[i]) if end is not None else 2 ** 40
            if e <= b:
                continue
            if e >= length:
                e = 2 ** 40
                if b < length:
                    self.len[s] = b
            for j in range(self.table_ld):
                if j * self.page >= b and (j + 1) * self.page <= e:
                    if self.names(self.table[s, j]):
                        self.refs[self.table[s, j]] -= 1
                    self.table[s, j] = -1

    def reserve(self, new):
        """(pages lacking, rows too short)"""
        asks, narrow = [], 0
        for s in range(self.n_seq):
            n, a = max(int(self.len[s]), 0), int(new[s])
            if a <= 0:
                continue
            last = (n + a - 1) // self.page
            if last >= self.table_ld:
                narrow += 1
                continue
            asks += [(s, j, n) for j in range(n // self.page, last + 1)]
        writers = {}
        for s, j, _ in asks:
            p = int(self.table[s, j])
            if self.names(p):
                writers.setdefault(p, []).append(s)
        todo = []
        for s, j, n in asks:
            p = int(self.table[s, j])
            if not self.names(p):
                todo.append((s, j, None, 0))
            elif self.refs[p] > 1 and not (len(writers[p]) == self.refs[p] and min(writers[p]) == s):
                todo.append((s, j, p, min(max(n - j * self.page, 0), self.page)))
        free = np.nonzero(self.refs <= 0)[0]
        short = max(len(todo) - len(free), 0)
        if short or narrow:
            return short, narrow
        for (s, j, p, count), q in zip(todo, free):
            self.table[s, j] = q
            self.refs[q] = 1
            if p is None:
                continue
            self.refs[p] -= 1
            if count:
                for codes, scales in zip(self.codes, self.scales):
                    for c, sc in zip(codes, scales):
                        c[q, :, :count] = c[p, :, :count]
                        sc[q] = sc[p]
        return 0, 0

    def compact(self):
        """(moved, pages in use)"""
        used = int((self.refs > 0).sum())
        src = [p for p in range(used, self.n_pages) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] <= 0]
        moved = np.where(self.refs > 0, np.arange(self.n_pages), -1).astype(np.int32)
        moved[src] = dst
        for p, q in zip(src, dst):
            self.refs[q], self.refs[p] = self.refs[p], 0
            for codes, scales in zip(self.codes, self.scales):
                for c, sc in zip(codes, scales):
                    c[q], sc[q] = c[p], sc[p]
        for e in np.nditer(self.table, op_flags=["readwrite"]):
            p = int(e)
            if self.names(p) and moved[p] >= 0:
                e[...] = moved[p]
        return moved, used
