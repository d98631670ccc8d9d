"""Plain 64-bit reference of the paged operators (tests only), written from their definitions on Python
lists and numpy arrays: page tables, and the norm before the rotation."""
import numpy as np


class Pages:
    """A page table as lists: rows of pages, lengths, and the stack of free pages."""

    def __init__(self, batch, width, page, pages):
        self.page, self.width, self.pages = page, width, pages
        self.rows, self.length = [[] for _ in range(batch)], [0] * batch
        self.free = list(range(pages - 1, -1, -1))

    def need(self, tokens):
        return -(-tokens // self.page)

    def update(self, keep, count, n):
        batch = len(self.rows)
        given = []
        for b in range(batch):
            if keep is not None:
                self.length[b] = min(self.length[b], max(0, keep[b]))
            k = self.need(self.length[b])
            given += self.rows[b][k:]
            del self.rows[b][k:]
        self.free += given[::-1]
        first, granted, slot, at = [], [], [-1] * n, [-1] * n
        row = asked = 0
        there = len(self.free)
        for b in range(batch):
            want = max(0, count[b]) if count is not None else 0
            first.append(min(row, 2 ** 31 - 1))
            ok = row + want <= n and self.length[b] + want <= self.width * self.page
            new = self.need(self.length[b] + want) - self.need(self.length[b]) if ok else 0
            asked += new
            ok = ok and (new == 0 or asked <= there)
            granted.append(want if ok else 0)
            if ok:
                self.rows[b] += [self.free.pop() for _ in range(new)]
                for i in range(want):
                    p = self.length[b] + i
                    at[row + i] = p
                    slot[row + i] = self.rows[b][p // self.page] * self.page + p % self.page
                self.length[b] += want
            row += want
        return first, granted, slot, at

    def table(self):
        return np.array([r + [-1] * (self.width - len(r)) for r in self.rows], np.int32)

    def stack(self):
        return np.array(self.free + [-1] * (self.pages - len(self.free)), np.int32)


def norm(x, w, eps):
    """Rows [n][128] float64 over the root of their mean square, times w."""
    with np.errstate(all="ignore"):
        return x / np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps) * w
