"""fp64 CPU oracle of rotary positions and a plain model of a cache's pages
(test infrastructure; shares nothing with the CUDA library)."""
from __future__ import annotations

import numpy as np


def rope(x, positions, inv_freq, rot_dim, rot_offset, pairing, inverse=False, mscale=1.0):
    """x [rows, N, D] float64, positions [rows], inv_freq [rot_dim/2]."""
    y = np.array(x, dtype=np.float64)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None]
    w = mscale * np.exp((-1j if inverse else 1j) * a)[:, None, :]
    o, h = rot_offset, rot_dim // 2
    i = np.arange(h)
    c0, c1 = (o + i, o + h + i) if pairing == "half" else (o + 2 * i, o + 2 * i + 1)
    z = (y[..., c0] + 1j * y[..., c1]) * w
    y[..., c0], y[..., c1] = z.real, z.imag
    return y


class Pages:
    """A cache's pages, one step at a time in plain Python.  ``flags`` collects
    the LI_DEV_* bits that the library documents."""

    NO_PAGES, BAD_ROW, BAD_KLEN, BAD_BLOCK = 0x40, 0x80, 0x02, 0x04

    def __init__(self, table, lens, refs, page_size, pools=()):
        self.table = [list(map(int, r)) for r in table]
        self.lens = [int(n) for n in lens]
        self.refs = [int(r) for r in refs]
        self.ps = page_size
        self.cols = len(self.table[0])
        self.pools = [np.array(p) for p in pools]
        self.flags = 0

    def _pages(self, n):
        return -(-n // self.ps)

    def _free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _clamp(self):
        cap = self.cols * self.ps
        for b, n in enumerate(self.lens):
            if n < 0 or n > cap:
                self.flags |= self.BAD_KLEN
                self.lens[b] = min(max(n, 0), cap)

    def _page(self, p):
        if 0 <= p < len(self.refs):
            return p
        self.flags |= self.BAD_BLOCK
        return -1

    def reserve(self, new_lens):
        self._clamp()
        free, used, open_ = self._free_pages(), 0, True
        for b, want in enumerate(map(int, new_lens)):
            if want < 0 or want > self.cols * self.ps:
                self.flags |= self.BAD_KLEN
                continue
            if want <= self.lens[b]:
                continue
            had, need = self._pages(self.lens[b]), self._pages(want) - self._pages(self.lens[b])
            used += need
            if need and used > len(free):
                self.flags |= self.NO_PAGES
                continue
            for j in range(need):
                p = free[used - need + j]
                self.table[b][had + j] = p
                self.refs[p] = 1
            self.lens[b] = want

    def fork(self, src, dst):
        self._clamp()
        free, used, taken, before = self._free_pages(), 0, set(), list(self.lens)
        for s, d in zip(map(int, src), map(int, dst)):
            B = len(before)
            if not (0 <= d < B and 0 <= s < B) or before[d] != 0 or d in taken:
                self.flags |= self.BAD_ROW
                continue
            taken.add(d)
            n = before[s]
            full, need = n // self.ps, int(n % self.ps != 0)
            used += need
            if need and used > len(free):
                self.flags |= self.NO_PAGES
                continue
            row = [self._page(p) for p in self.table[s][:full]]
            if need:
                p = free[used - 1]
                old = self._page(self.table[s][full])
                if old >= 0:
                    for pool in self.pools:
                        pool[p] = pool[old]
                row.append(p)
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
            self.table[d] = row + [-1] * (self.cols - len(row))
            self.lens[d] = n

    def free(self, rows):
        self._clamp()
        done = set()
        for r in map(int, rows):
            if not 0 <= r < len(self.lens) or r in done:
                self.flags |= self.BAD_ROW
                continue
            done.add(r)
            for c in range(self._pages(self.lens[r])):
                p = self._page(self.table[r][c])
                if p >= 0:
                    if self.refs[p] <= 0:
                        self.flags |= self.BAD_BLOCK
                    else:
                        self.refs[p] -= 1
            self.table[r] = [-1] * self.cols
            self.lens[r] = 0

    def compact(self):
        self._clamp()
        n = sum(r != 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in range(n, len(self.refs)) if self.refs[p] != 0]
        to = dict(zip(movers, holes))
        for r, row in enumerate(self.table):
            for c in range(self.cols):
                p = self._page(row[c]) if c < self._pages(self.lens[r]) else -1
                row[c] = to.get(p, p)
        for m, h in to.items():
            self.refs[h], self.refs[m] = self.refs[m], 0
            for pool in self.pools:
                pool[h] = pool[m]
