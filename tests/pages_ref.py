"""A pool of pages and a block table on the host, entry by entry: what the page operators make of them. No code shared with
the library. Each call returns the status bits that it raises."""

import numpy as np

BOUNDS, NO_PAGES = 8, 32


class Pool:
    def __init__(self, page_size, num_pages, rows, columns):
        self.page, self.pages, self.columns = page_size, num_pages, columns
        self.refs = np.zeros(num_pages, np.int32)
        self.table = np.full((rows, columns), -1, np.int32)
        self.planes = []  # [pages, vectors, page_size, ...]

    def _listed(self, rows):
        """The listed rows that count, each with its place in the list."""
        got, status, seen = [], 0, set()
        for i, r in enumerate(rows):
            if r < 0 or r >= len(self.table) or r in seen:
                status |= BOUNDS
            else:
                got.append((i, int(r)))
            seen.add(r)
        return got, status

    def _free(self):
        return iter(np.flatnonzero(self.refs == 0).tolist())

    def _give_back(self, pages):
        status = 0
        for x in pages:
            if x >= self.pages or self.refs[x] <= 0:
                status |= BOUNDS
            else:
                self.refs[x] -= 1
        return status

    def resize(self, end, begin=None, keep_first=0, rows=None):
        listed, status = self._listed(range(len(end)) if rows is None else rows)
        cap, free, dropped, taken = self.columns * self.page, self._free(), [], []
        for i, r in listed:
            b, e = 0 if begin is None else int(begin[i]), int(end[i])
            if b > cap or e > cap:
                status |= BOUNDS
            b, e = min(max(b, 0), cap), min(max(e, 0), cap)
            for c in range(self.columns):
                first = c * self.page
                last = first + self.page
                want = first < e and (last > b or first < min(keep_first, e))
                if want and self.table[r, c] < 0:
                    page = next(free, None)
                    if page is None:
                        status |= NO_PAGES
                    else:
                        self.table[r, c] = page
                        taken.append(page)
                elif not want and self.table[r, c] >= 0:
                    dropped.append(self.table[r, c])
                    self.table[r, c] = -1
        for x in taken:
            self.refs[x] += 1
        return status | self._give_back(dropped)

    def fork(self, src, dst, length):
        listed, status = self._listed(dst)
        was, free, dropped, held, moves = self.table.copy(), self._free(), [], [], []
        counts = self.refs.copy()
        cap = self.columns * self.page
        for i, r in listed:
            a = int(src[i])
            if a < 0 or a >= len(self.table):
                status |= BOUNDS
                continue
            if a == r:
                continue
            n = int(length[i])
            if n > cap:
                status |= BOUNDS
            n = min(max(n, 0), cap)
            dropped += [x for x in was[r] if x >= 0]
            for c in range(self.columns):
                self.table[r, c] = -1
                x = was[a, c]
                if c * self.page >= n or x < 0:
                    continue
                if x >= self.pages or counts[x] <= 0:
                    status |= BOUNDS
                    continue
                rest = n - c * self.page
                if rest >= self.page:
                    self.table[r, c] = x
                    held.append(x)
                else:
                    page = next(free, None)
                    if page is None:
                        status |= NO_PAGES
                        continue
                    self.table[r, c] = page
                    held.append(page)
                    moves.append((x, page, rest))
        for x in held:
            self.refs[x] += 1
        status |= self._give_back(dropped)
        for x, page, rest in moves:
            for plane in self.planes:
                plane[page][:, :rest] = plane[x][:, :rest]
        return status

    def compact(self, start, keep, rows=None):
        listed, status = self._listed(range(len(start)) if rows is None else rows)
        moves = []
        for i, r in listed:
            ids = []
            for x in keep[i]:
                if x < 0:
                    break
                ids.append(int(x))
            s, row = int(start[i]), []
            ok = not ids or (s >= 0 and ids[0] >= s and all(a < b for a, b in zip(ids, ids[1:])))
            ok = ok and all(x // self.page < self.columns for x in ids)
            if ok:
                for j, x in enumerate(ids):
                    a, b = self.table[r, x // self.page], self.table[r, (s + j) // self.page]
                    if not (0 <= a < self.pages and 0 <= b < self.pages) or (x != s + j and self.refs[b] > 1):
                        ok = False
                    row.append((a, x % self.page, b, (s + j) % self.page))
            if ok:
                moves += row
            else:
                status |= BOUNDS
        for plane in self.planes:
            new = [plane[a][:, ta].copy() for a, ta, _, _ in moves]
            for (_, _, b, tb), x in zip(moves, new):
                plane[b][:, tb] = x
        return status
