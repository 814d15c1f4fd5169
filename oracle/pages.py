"""Oracle of the page pool (include/ccb_pages.h): trim and grow with Python
lists, one sequence and page at a time.  Shares no code with the library."""

from __future__ import annotations


class Pool:
    """free: the stack (its unused part too), count: how many are in use,
    table: a list of page numbers for each sequence, lens: their tokens."""

    def __init__(self, page_size, free, count, table, lens):
        self.page, self.free, self.count = page_size, list(free), count
        self.table, self.lens = [list(row) for row in table], list(lens)
        self.bad = False

    def _pages(self, tokens):
        return -(-tokens // self.page)

    def _number(self, page):
        if not 0 <= page < len(self.free):
            self.bad = True
            return -1
        return page

    def trim(self, keep):
        room = len(self.table[0]) * self.page if self.table else 0
        after, back = [], []
        for n, k, row in zip(self.lens, keep, self.table):
            if not 0 <= n <= room:
                self.bad = True
                after.append(n)
                continue
            left = n if k < 0 else min(n, k)
            after.append(left)
            back += row[self._pages(left):self._pages(n)]
        if not 0 <= self.count or self.count + len(back) > len(self.free):
            self.bad = True
            return
        for page in reversed(back):
            self.free[self.count] = self._number(page)
            self.count += 1
        self.lens = after

    def grow(self, counts, tokens):
        """Returns slots, positions, sequences, starts, granted."""
        room = len(self.table[0]) * self.page if self.table else 0
        slots, positions, sequences = [-1] * tokens, [-1] * tokens, [-1] * tokens
        starts, granted, at = [], [], 0
        sound = 0 <= self.count <= len(self.free)
        have = left = self.count if sound else 0  # left: were everybody served
        self.bad |= not sound
        taken = 0
        for b, (n, c) in enumerate(zip(list(self.lens), counts)):
            starts.append(min(at, tokens))
            asks = max(c, 0)
            ok = c >= 0 and 0 <= n <= room and n + c <= room and at + asks <= tokens
            self.bad |= not ok
            need = self._pages(n + c) - self._pages(n) if ok else 0
            left -= need
            fits = ok and (need == 0 or left >= 0)
            if fits:
                for j in range(self._pages(n), self._pages(n + c)):
                    taken += 1
                    self.table[b][j] = self.free[have - taken]
                self.lens[b] = n + c
            granted.append(c if fits else 0)
            for i in range(at, min(at + asks, tokens)):
                sequences[i] = b
                if fits:
                    t = n + i - at
                    page = self._number(self.table[b][t // self.page])
                    positions[i] = t
                    slots[i] = page * self.page + t % self.page if page >= 0 else -1
            at += asks
        starts.append(min(at, tokens))
        if sound:
            self.count = have - taken
        return slots, positions, sequences, starts, granted
