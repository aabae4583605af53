"""A plain model of the page calls: table rows, counts and lengths changed row by row, with
token contents as tags, so that a test can say what every token of every sequence must be."""
from __future__ import annotations


class Pages:
    def __init__(self, B: int, max_pages: int, num_pages: int, P: int):
        self.B, self.max_pages, self.num_pages, self.P = B, max_pages, num_pages, P
        self.rows = [[-1] * max_pages for _ in range(B)]
        self.refs = [0] * num_pages
        self.lens = [0] * B
        self.info = [0] * 4

    def _free(self):
        return [i for i, r in enumerate(self.refs) if r <= 0]

    def _in_use(self):
        return sum(r > 0 for r in self.refs)

    def _held(self, page):
        return 0 <= page < self.num_pages

    def reserve(self, extra):
        free, got, missing = self._free(), 0, 0
        for b, e in enumerate(extra):
            if e <= 0:
                continue
            want = min(max(self.lens[b], 0) + e, self.max_pages * self.P)
            for j in range(-(-want // self.P)):
                if self._held(self.rows[b][j]):
                    continue
                self.rows[b][j] = -1
                if got < len(free):
                    self.rows[b][j] = free[got]
                    self.refs[free[got]] = 1
                    got += 1
                else:
                    missing += 1
        self.info = [got, missing, self._in_use(), 0]

    def reorder(self, parent):
        """Returns [(b, source, page copied from, page copied to)] of the changed, nonempty rows."""
        B, P = self.B, self.P
        parent = [p if 0 <= p < B else -1 for p in parent]
        lens = [min(max(n, 0), self.max_pages * P) for n in self.lens]
        clean = [[x if self._held(x) else -1 for x in row] for row in self.rows]
        heir = {}
        for s in range(B):
            copies = [b for b in range(B) if parent[b] == s]
            if copies:
                heir[s] = s if s in copies else copies[0]
        before = self._in_use()
        new, split = {}, []
        for b, s in enumerate(parent):
            if s == b:
                continue
            if s < 0:
                new[b] = [-1] * self.max_pages
            elif heir[s] == b:
                new[b] = list(clean[s])
            else:
                full = lens[s] // P
                new[b] = clean[s][:full] + [-1] * (self.max_pages - full)
                if lens[s] % P and clean[s][full] >= 0:
                    split.append(b)
        for b in new:
            for x in clean[b]:
                if x >= 0:
                    self.refs[x] -= 1
            for x in new[b]:
                if x >= 0:
                    self.refs[x] += 1
        given_back = before - self._in_use()
        free, got, copied = self._free(), 0, {}
        for b in new:
            self.lens[b] = lens[parent[b]] if parent[b] >= 0 else 0
        for b in split:
            full = lens[parent[b]] // P
            if got < len(free):
                copied[b] = (clean[parent[b]][full], free[got])
                new[b][full] = free[got]
                self.refs[free[got]] = 1
                got += 1
            else:
                self.lens[b] = full * P
        for b in new:
            self.rows[b] = new[b]
        self.info = [got, len(split) - got, self._in_use(), given_back]
        return [(b, parent[b], *copied.get(b, (-1, -1))) for b in new if parent[b] >= 0]

    def compact(self):
        """Returns the new id of every page."""
        live = [i for i, r in enumerate(self.refs) if r > 0]
        L = len(live)
        holes = [i for i in range(L) if self.refs[i] <= 0]
        movers = [i for i in live if i >= L]
        new = [-1] * self.num_pages
        for i in live:
            new[i] = i
        for m, h in zip(movers, holes):
            new[m] = h
        refs = [0] * self.num_pages
        for i in live:
            refs[new[i]] = self.refs[i]
        self.rows = [[new[x] if self._held(x) else -1 for x in row] for row in self.rows]
        self.refs, self.info = refs, [len(movers), 0, L, 0]
        return new
