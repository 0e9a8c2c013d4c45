"""Forking, growing, trimming and compacting sequences over a pool of pages, one after the other in plain Python
(test infrastructure only). Every rule is the text of include/cp.h."""
from __future__ import annotations

import numpy as np


class Pool:
    def __init__(self, refs, table, length, page_size):
        self.refs, self.table, self.length = (np.array(a, np.int64) for a in (refs, table, length))
        self.page, self.bad = page_size, False

    def held(self, length):
        return -(-int(length) // self.page)

    def len_of(self, i):
        n = int(self.length[i])
        if 0 <= n and self.held(n) <= self.table.shape[1]:
            return n
        self.bad = True
        return 0

    def ok(self, page):
        return 0 <= page < len(self.refs)

    def fork(self, src, dst):
        n = len(self.length)
        before = self.length.copy()
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < n and 0 <= d < n) or list(dst).count(d) > 1 or d in list(src) or before[d] != 0:
                self.bad = True
                continue
            length = self.len_of(s)
            if any(self.ok(page) and self.refs[page] < 1 for page in self.table[s, : self.held(length)]):
                self.bad = True
                continue
            self.length[d] = length
            for k in range(self.held(length)):
                page = self.table[s, k]
                self.table[d, k] = page
                if self.ok(page):
                    self.refs[page] += 1
                else:
                    self.bad = True

    def trim(self, keep):
        for i, want in enumerate(keep):
            length = self.len_of(i)
            if want < 0:
                self.bad = True
            elif want < length:
                for k in range(self.held(want), self.held(length)):
                    page = self.table[i, k]
                    self.table[i, k] = -1
                    if self.ok(page) and self.refs[page] > 0:
                        self.refs[page] -= 1
                    else:
                        self.bad = True
                self.length[i] = want

    def grow(self, add):
        """(moves, count)."""
        grows, sharers = [], {}
        for i, more in enumerate(add):
            length = self.len_of(i)
            if more == 0 or length != self.length[i]:
                continue
            if more < 0 or length + more > 2 ** 31 - 1 or self.held(length + more) > self.table.shape[1]:
                self.bad = True
                continue
            last = -1
            if length % self.page:
                page = self.table[i, self.held(length) - 1]
                if not self.ok(page) or self.refs[page] < 1:
                    self.bad = True
                    continue
                last = int(page)
                sharers.setdefault(last, []).append(i)
            grows.append((i, length, int(length + more), last))
        short = {p for p, who in sharers.items() if len(who) > self.refs[p]}
        self.bad |= len(short) > 0
        grows = [g for g in grows if g[3] not in short]
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        plan, need = [], 0
        for i, length, to, last in grows:
            stays = last >= 0 and len(sharers[last]) == self.refs[last] and sharers[last][-1] == i
            copies = last >= 0 and not stays
            plan.append((i, length, to, last, copies))
            need += self.held(to) - self.held(length) + copies
        if need > len(free):
            return [], len(free) - need
        moves, take = [], iter(free)
        for i, length, to, last, copies in plan:
            if copies:
                page = next(take)
                moves.append((last, page))
                self.table[i, self.held(length) - 1] = page
                self.refs[page] += 1
                self.refs[last] -= 1
            for k in range(self.held(length), self.held(to)):
                page = next(take)
                self.table[i, k] = page
                self.refs[page] += 1
            self.length[i] = to
        return moves, len(moves)

    def compact(self):
        n = int((self.refs != 0).sum())
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in range(n, len(self.refs)) if self.refs[p] != 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for i in range(len(self.length)):
            for k in range(self.held(self.len_of(i))):
                page = int(self.table[i, k])
                if not self.ok(page) or page in holes or page >= n and page not in to:
                    self.bad = True
                elif page >= n:
                    self.table[i, k] = to[page]
        return list(to.items()), len(to)
