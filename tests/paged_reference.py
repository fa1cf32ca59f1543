"""Plain implementations in 64 bits of the paged-cache operators (numpy, one
sequence, head and row at a time), for the tests."""
from __future__ import annotations

import numpy as np


def ancestors(parents):
    """sees[i] = the nodes on the way from node i to the root, i first."""
    sees = []
    for i, p in enumerate(parents):
        sees.append([i] + (sees[p] if p >= 0 else []))
    return sees


def mask_words(parents, live):
    """(words int32 [T][ceil(T/32)], depth int32 [T]) of one tree."""
    T = len(parents)
    words = np.zeros((T, (T + 31) // 32), np.uint32)
    depth = np.zeros(T, np.int32)
    for i, s in enumerate(ancestors(parents)):
        if i < live:
            for j in s:
                words[i, j // 32] |= np.uint32(1 << (j % 32))
            depth[i] = len(s) - 1
    return words.view(np.int32), depth


def tree_rows(q, k, v, k_tree, v_tree, sees, scale):
    """One unit: q [g][T][d], cached k, v [n][d], tree rows [t][d], sees [T][t]
    truth values.  Returns out [g][T][d], lse2 [g][T] and a [g][T][d] = the
    weights' sum of |v|, which the tolerances use."""
    g, T, d = q.shape
    out, mag = np.zeros((g, T, d)), np.zeros((g, T, d))
    lse2 = np.full((g, T), -np.inf)
    n = k.shape[0]
    for h in range(g):
        for i in range(T):
            nodes = np.flatnonzero(sees[i]) if k_tree is not None else np.zeros(0, int)
            kk = np.concatenate([k, k_tree[nodes]]) if len(nodes) else k
            vv = np.concatenate([v, v_tree[nodes]]) if len(nodes) else v
            if kk.shape[0] == 0:
                continue
            z = scale * (kk @ q[h, i])
            m = z.max()
            w = np.exp(z - m)
            s = w.sum()
            out[h, i] = (w / s) @ vv
            mag[h, i] = (w / s) @ np.abs(vv)
            lse2[h, i] = (m + np.log(s)) / np.log(2.0)
    assert n == k.shape[0]
    return out, lse2, mag


class Book:
    """The page table, lengths and reference counts, by the definition."""

    def __init__(self, n_pages, n_seqs, max_pages, page_rows):
        self.refs = [0] * n_pages
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.lens = [0] * n_seqs
        self.page, self.max_pages = page_rows, max_pages
        self.copies = []                    # (from, to, rows) of the last reserve

    def state(self):
        return [list(self.refs), [list(r) for r in self.table], list(self.lens)]

    def restore(self, st):
        self.refs, self.table, self.lens = st

    def _pages(self, rows):
        return -(-rows // self.page)

    def _take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def reserve(self, seqs, n_new):
        self.copies = []
        if len(set(seqs)) < len(seqs) or any(s < 0 or s >= len(self.lens) for s in seqs) or any(x < 0 for x in n_new) \
                or any(self.lens[s] + x > self.max_pages * self.page for s, x in zip(seqs, n_new)):
            return -1
        before, want, leavers = self.state(), 0, {}
        for s, x in zip(seqs, n_new):
            n = self.lens[s]
            if x and n % self.page:
                tail = self.table[s][n // self.page]
                if self.refs[tail] - leavers.get(tail, 0) > 1:
                    leavers[tail] = leavers.get(tail, 0) + 1
                    want += 1
            want += self._pages(n + x) - self._pages(n)
        if want > self.refs.count(0):
            return want - self.refs.count(0)
        for s, x in zip(seqs, n_new):
            n = self.lens[s]
            at = n // self.page
            if x and n % self.page and self.refs[self.table[s][at]] > 1:
                old = self.table[s][at]
                self.table[s][at] = self._take()
                self.refs[old] -= 1
                self.copies.append((old, self.table[s][at], n % self.page))
            for p in range(self._pages(n), self._pages(n + x)):
                self.table[s][p] = self._take()
            self.lens[s] = n + x
        del before
        return 0

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            n = min(self.lens[s], 0 if keep is None else keep[i])
            for p in range(self._pages(n), self.max_pages):
                if self.table[s][p] >= 0:
                    self.refs[self.table[s][p]] -= 1
                    self.table[s][p] = -1
            self.lens[s] = n

    def fork(self, src, dst, n_rows=None):
        if len(set(dst)) < len(dst):
            return -1
        old = self.state()
        for i, (a, b) in enumerate(zip(src, dst)):
            n = old[2][a] if n_rows is None else min(old[2][a], n_rows[i])
            new = [p if x < self._pages(n) else -1 for x, p in enumerate(old[1][a])]
            for p in new:
                if p >= 0:
                    self.refs[p] += 1
            for p in old[1][b]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[b], self.lens[b] = new, n
        return 0

    def compact(self, src, dst, n_idx):
        """Returns (result, the sources' old tables)."""
        if len(set(dst)) < len(dst):
            return -1, None
        old = self.state()
        for a in src:
            for p in old[1][a]:
                if p >= 0:
                    self.refs[p] += 1
        for b in dst:
            for p in old[1][b]:
                if p >= 0:
                    self.refs[p] -= 1
        per = self._pages(n_idx)
        if len(src) * per > self.refs.count(0):
            missing = len(src) * per - self.refs.count(0)
            self.restore(old)
            return missing, None
        for b in dst:
            self.table[b] = [self._take() if x < per else -1 for x in range(self.max_pages)]
            self.lens[b] = n_idx
        for a in src:
            for p in old[1][a]:
                if p >= 0:
                    self.refs[p] -= 1
        return 0, [old[1][a] for a in src]
