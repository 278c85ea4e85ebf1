"""The attention cache's rules on plain lists (test infrastructure): which pages each call takes,
shares, gives back and renumbers."""


class Model:
    def __init__(self, rows, max_pages, pages, page):
        self.page, self.max_pages = page, max_pages
        self.rows = [[] for _ in range(rows)]
        self.lengths = [0] * rows
        self.refs = [0] * pages

    def held(self, n):
        return -(-n // self.page)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, counts):
        free, used, start = self.free_pages(), 0, []
        for r, n in enumerate(counts):
            to = self.held(self.lengths[r] + n) if n >= 0 else 0
            if n < 0 or to > self.max_pages:
                start.append(-1)
                continue
            need = to - len(self.rows[r])
            used += need          # a row that fails leaves nothing for those behind it
            if need and used > len(free):
                start.append(-1)
                continue
            start.append(self.lengths[r])
            got = free[used - need:used]
            for p in got:
                self.refs[p] = 1
            self.rows[r] += got
            self.lengths[r] += n
        return start

    def free(self, rows):
        for r in rows:
            if 0 <= r < len(self.rows):
                for p in self.rows[r]:
                    self.refs[p] -= 1
                self.rows[r], self.lengths[r] = [], 0

    def fork(self, src, dst):
        """Returns the copies (old page, new page, tokens)."""
        free, used, seen, copies, todo = self.free_pages(), 0, set(), [], []
        n = len(self.rows)
        for a, b in zip(src, dst):
            if not (0 <= a < n and 0 <= b < n) or self.lengths[b] or b in seen:
                continue
            seen.add(b)
            length = self.lengths[a]
            full, tail = length // self.page, length % self.page
            used += tail > 0
            if tail and used > len(free):
                continue
            todo.append((b, self.rows[a][:full], length, free[used - 1] if tail else None))
            if tail:
                copies.append((self.rows[a][full], free[used - 1], tail))
        for b, shared, length, fresh in todo:
            for p in shared:
                self.refs[p] += 1
            if fresh is not None:
                self.refs[fresh] = 1
            self.rows[b] = list(shared) + ([fresh] if fresh is not None else [])
            self.lengths[b] = length
        return copies

    def compact(self, pages):
        """Returns the old numbers of the pages in their new order (None: no room)."""
        live = [p for p, r in enumerate(self.refs) if r > 0]
        if len(live) > pages:
            return None
        number = {p: i for i, p in enumerate(live)}
        self.rows = [[number[p] for p in r] for r in self.rows]
        self.refs = [self.refs[p] for p in live] + [0] * (pages - len(live))
        return live

    def table(self):
        return [r + [-1] * (self.max_pages - len(r)) for r in self.rows]
