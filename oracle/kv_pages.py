"""The paged cache by its definition: one sequence after the other, plain
lists. Rows are opaque values (whatever a test writes into them)."""
from __future__ import annotations


class Pages:
    def __init__(self, n_pages, page_size, max_seqs, max_pages):
        self.size, self.max_pages = page_size, max_pages
        self.rows = [[None] * page_size for _ in range(n_pages)]
        self.refs = [0] * n_pages
        self.table = [[] for _ in range(max_seqs)]
        self.length = [0] * max_seqs

    def _take(self):
        page = self.refs.index(0)
        self.refs[page] = 1
        return page

    def extend(self, seqs, add):
        """False (and nothing changed) where it cannot be done as a whole."""
        if len(set(seqs)) < len(seqs):
            return False
        want, shared = 0, list(self.refs)
        for s, a in zip(seqs, add):
            pages = -(-(self.length[s] + a) // self.size)
            if pages > self.max_pages:
                return False
            want += pages - len(self.table[s])
            if a > 0 and self.length[s] % self.size and shared[self.table[s][-1]] > 1:
                shared[self.table[s][-1]] -= 1
                want += 1
        if want > self.refs.count(0):
            return "pages"
        given = []  # all pages are taken first: an open page that is left never becomes free
        for s, a in zip(seqs, add):
            if a > 0 and self.length[s] % self.size and self.refs[self.table[s][-1]] > 1:
                old, new = self.table[s][-1], self._take()
                self.refs[old] -= 1
                self.table[s][-1] = new
                given.append((old, new, self.length[s] % self.size))
            self.length[s] += a
            while len(self.table[s]) * self.size < self.length[s]:
                self.table[s].append(self._take())
        for old, new, n in given:
            self.rows[new][:n] = self.rows[old][:n]
        return True

    def write(self, s, pos, value):
        page = self.table[s][pos // self.size]
        if self.refs[page] != 1:
            return False
        self.rows[page][pos % self.size] = value
        return True

    def read(self, s, pos):
        return self.rows[self.table[s][pos // self.size]][pos % self.size]

    def fork(self, src, dst):
        self.table[dst], self.length[dst] = list(self.table[src]), self.length[src]
        for p in self.table[dst]:
            self.refs[p] += 1

    def truncate(self, s, to):
        self.length[s] = min(self.length[s], to)
        while len(self.table[s]) * self.size >= self.length[s] + self.size:
            self.refs[self.table[s].pop()] -= 1

    def keep(self, s, drafted, places):
        start = self.length[s] - drafted
        if places and any(self.refs[p] != 1 for p in self.table[s][start // self.size:]):
            return False
        values = [self.read(s, start + x) for x in places]
        for j, value in enumerate(values):
            self.write(s, start + j, value)
        self.truncate(s, start + len(places))
        return True

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        src = [p for p in range(used, len(self.refs)) if self.refs[p]]
        dst = [p for p in range(used) if not self.refs[p]]
        for a, b in zip(src, dst):
            self.rows[b], self.refs[b], self.refs[a] = list(self.rows[a]), self.refs[a], 0
        to = dict(zip(src, dst))
        self.table = [[to.get(p, p) for p in t] for t in self.table]
