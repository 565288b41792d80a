"""Plain definitions (numpy) of free, trim, fork and compact, and random
states of a cache's pages."""
from __future__ import annotations

import numpy as np


class Pages:
    """ctx, table, held, ring, state, extra as arrays; k, v [layers][P][H][page][D]
    arrays or None."""

    FIELDS = ("ctx", "table", "held", "ring", "state", "extra")

    def __init__(self, batch, P, page, width, head=0):
        self.P, self.page, self.width, self.batch = P, page, width, batch
        self.ctx = np.zeros(batch, np.int32)
        self.table = np.full((batch, width), -1, np.int32)
        self.held = np.zeros(batch, np.int32)
        self.ring = np.roll(np.arange(P), head).astype(np.int32)
        self.state = np.array([head, P], np.int32)
        self.extra = np.zeros(P, np.int32)
        self.k = self.v = None

    def take(self):
        head, count = self.state
        assert count > 0
        p = int(self.ring[head])
        self.state[:] = (head + 1) % self.P, count - 1
        return p

    def grow(self, b, tokens):
        """Give request b the pages of so many positions and that context."""
        self.ctx[b] = tokens
        while self.held[b] * self.page < tokens:
            self.table[b, self.held[b]] = self.take()
            self.held[b] += 1

    def _let_go(self, pairs):
        gone = set()
        for b, keep in pairs:
            for j in range(keep, self.held[b]):
                p = int(self.table[b, j])
                self.table[b, j] = -1
                if not 0 <= p < self.P:
                    continue
                if self.extra[p] == 0:
                    gone.add(p)
                else:
                    self.extra[p] -= 1
            self.held[b] = min(self.held[b], keep)
        head, count = self.state
        for i, p in enumerate(sorted(gone)):
            self.ring[(head + count + i) % self.P] = p
        self.state[1] = count + len(gone)

    def free(self, places):
        on = [int(b) for b in places if 0 <= b < self.batch]
        self._let_go((b, 0) for b in dict.fromkeys(on))
        self.ctx[on] = 0

    def trim(self, n, N):
        n = np.clip(n, -1, N)
        need = -(-(np.maximum(self.ctx, 0).astype(np.int64) + n + 1)
                 // self.page)
        self._let_go((b, int(min(need[b], self.held[b])))
                     for b in range(self.batch))

    def fork(self, src, dst, length=None):
        ctx, held, table = self.ctx.copy(), self.held.copy(), self.table.copy()
        head, count = (int(x) for x in self.state)
        done, named, wanted, taken = [], set(), 0, 0
        for i, (s, d) in enumerate(zip(src, dst)):
            s, d = int(s), int(d)
            first = d not in named
            named.add(d)
            ok = (0 <= s < self.batch and 0 <= d < self.batch and s != d
                  and first and held[d] == 0)
            if ok:
                n = int(ctx[s])
                if length is not None:
                    n = min(n, max(int(length[i]), 0))
                full, rest = divmod(n, self.page)
                ok = full + (rest > 0) <= held[s]
            if ok and rest > 0:
                ok = 0 <= table[s, full] < self.P
            if ok and rest > 0:
                wanted += 1
                ok = wanted <= count
            done.append(int(ok))
            if not ok:
                continue
            self.ctx[d], self.held[d] = n, full + (rest > 0)
            self.table[d, :full] = table[s, :full]
            for p in table[s, :full]:
                if 0 <= p < self.P:
                    self.extra[p] += 1
            if rest > 0:
                p = int(self.ring[(head + wanted - 1) % self.P])
                self.table[d, full] = p
                taken = wanted
                for c in (self.k, self.v):
                    if c is not None:
                        c[:, p, :, :rest] = c[:, table[s, full], :, :rest]
        self.state[:] = (head + taken) % self.P, count - taken
        return np.array(done, np.int32)

    def compact(self):
        holders = np.zeros(self.P, np.int64)
        for b in range(self.batch):
            for p in self.table[b, :self.held[b]]:
                if 0 <= p < self.P:
                    holders[p] += 1
        T = int((holders > 0).sum())
        holes = [p for p in range(T) if holders[p] == 0]
        high = [p for p in range(T, self.P) if holders[p] > 0]
        to = np.arange(self.P)
        extra = np.maximum(holders - 1, 0)
        for a, b in zip(high, holes):
            to[a] = b
            extra[b], extra[a] = extra[a], 0
            for c in (self.k, self.v):
                if c is not None:
                    c[:, b] = c[:, a]
        for b in range(self.batch):
            for j in range(self.held[b]):
                if 0 <= self.table[b, j] < self.P:
                    self.table[b, j] = to[self.table[b, j]]
        self.extra[:] = extra
        self.ring[:] = (T + np.arange(self.P)) % self.P
        self.state[:] = 0, self.P - T


def check(s):
    """Every page is free or held, and counted right."""
    head, count = s.state
    free = [int(s.ring[(head + i) % s.P]) for i in range(count)]
    holders = np.zeros(s.P, np.int64)
    for b in range(s.batch):
        assert (s.table[b, s.held[b]:] == -1).all()
        for p in s.table[b, :s.held[b]]:
            holders[p] += 1
    assert len(set(free)) == count and not holders[free].any()
    assert count + (holders > 0).sum() == s.P
    assert np.array_equal(s.extra, np.maximum(holders - 1, 0))
