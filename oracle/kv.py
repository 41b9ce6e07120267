"""Paged key/value cache and its attention in exact integers and fp64.

Written from the definitions, one head and one query at a time, on plain numpy
arrays and Python lists; shares no code with the library.  The layouts are the
library's (include/ft_kv.h): pool [n_pages][L][2][Hkv][page][D], table
[n_rows][row_pages] with -1 past a row's pages, lens [n_rows], refs [n_pages].
"""
from __future__ import annotations

import numpy as np


class Refused(Exception):
    """The call must change nothing: 'device' (a bad argument) or 'capacity' (too few free pages)."""


class Pages:
    """The control state, as lists of Python integers, and the list of page copies each call asks for."""

    def __init__(self, n_pages, n_rows, row_pages, page):
        self.n_pages, self.n_rows, self.row_pages, self.page = n_pages, n_rows, row_pages, page
        self.rows = [[] for _ in range(n_rows)]
        self.lens = [0] * n_rows
        self.refs = [0] * n_pages

    def _free_pages(self, want):
        got = [p for p in range(self.n_pages) if self.refs[p] == 0][:want]
        if len(got) < want:
            raise Refused("capacity")
        return got

    def _check_rows(self, rows):
        if len(set(rows)) != len(rows) or any(r < 0 or r >= self.n_rows for r in rows):
            raise Refused("device")

    def extend(self, rows, add):
        self._check_rows(rows)
        if any(a < 0 or self.lens[r] + a > self.row_pages * self.page for r, a in zip(rows, add)):
            raise Refused("device")
        need = [-(-(self.lens[r] + a) // self.page) - len(self.rows[r]) for r, a in zip(rows, add)]
        got = self._free_pages(sum(need))
        for r, a, n in zip(rows, add, need):
            for _ in range(n):
                p = got.pop(0)
                self.rows[r].append(p)
                self.refs[p] = 1
            self.lens[r] += a
        return []

    def fork(self, parents, children):
        self._check_rows(children)
        if (any(p < 0 or p >= self.n_rows for p in parents) or any(self.lens[c] for c in children)
                or set(parents) & set(children)):
            raise Refused("device")
        got = self._free_pages(sum(1 for p in parents if self.lens[p] % self.page))
        copies = []
        for p, c in zip(parents, children):
            full, part = divmod(self.lens[p], self.page)
            new = list(self.rows[p][:full])
            for x in new:
                self.refs[x] += 1
            if part:
                x = got.pop(0)
                self.refs[x] = 1
                copies.append((self.rows[p][full], x, part))
                new.append(x)
            self.rows[c], self.lens[c] = new, self.lens[p]
        return copies

    def reorder(self, rows, parents):
        self._check_rows(rows)
        if any(p < -1 or p >= self.n_rows for p in parents):
            raise Refused("device")
        old_rows, old_lens, old_refs = [list(r) for r in self.rows], list(self.lens), list(self.refs)
        # which item keeps its parent's incomplete page: the parent's own row, else the first in the list
        keeper = {}
        for i, (r, p) in enumerate(zip(rows, parents)):
            if p in rows and (p == r or p not in keeper):
                keeper[p] = i
        new, wanting = [], []
        for i, p in enumerate(parents):
            full, part = divmod(old_lens[p], self.page) if p >= 0 else (0, 0)
            pages = list(old_rows[p][:full]) if p >= 0 else []
            if part and keeper.get(p) == i:
                pages.append(old_rows[p][full])
            elif part:
                wanting.append((i, old_rows[p][full], part))
            new.append(pages)
        for r in rows:
            for x in old_rows[r]:
                self.refs[x] -= 1
        for pages in new:
            for x in pages:
                self.refs[x] += 1
        try:
            got = self._free_pages(len(wanting))
        except Refused:
            self.refs = old_refs
            raise
        copies = []
        for (i, src, part), x in zip(wanting, got):
            new[i].append(x)
            self.refs[x] = 1
            copies.append((src, x, part))
        for r, p, pages in zip(rows, parents, new):
            self.rows[r], self.lens[r] = pages, old_lens[p] if p >= 0 else 0
        return copies

    def batch(self, rows, add, T):
        """extend, and the lists of its new tokens: (cu_q, row_of, pos, slots), padded to T."""
        if any(a < 0 for a in add) or sum(add) > T:
            raise Refused("device")
        old = [self.lens[r] if 0 <= r < self.n_rows else 0 for r in rows]
        self.extend(rows, add)
        cu, row_of, pos, slots = [0], [], [], []
        for r, a, n in zip(rows, add, old):
            cu.append(cu[-1] + a)
            for i in range(n, n + a):
                row_of.append(r)
                pos.append(i)
                slots.append(self.rows[r][i // self.page] * self.page + i % self.page)
        pad = T - len(pos)
        return cu, row_of + [-1] * pad, pos + [0] * pad, slots + [-1] * pad

    def free(self, rows):
        self._check_rows(rows)
        for r in rows:
            for p in self.rows[r]:
                self.refs[p] -= 1
            self.rows[r], self.lens[r] = [], 0
        return []

    def compact(self):
        live = sum(1 for x in self.refs if x > 0)
        src = [p for p in range(live, self.n_pages) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return [(s, d, self.page) for s, d in to.items()]

    def table(self):
        t = np.full((self.n_rows, self.row_pages), -1, dtype=np.int32)
        for r, pages in enumerate(self.rows):
            t[r, :len(pages)] = pages
        return t


def copy_pages(pool, copies):
    """Apply copies (src, dst, tokens) to pool [n_pages, L, 2, Hkv, page, D] in place."""
    for s, d, tok in copies:
        pool[d, :, :, :, :tok] = pool[s, :, :, :, :tok]


def normed(x, w, eps):
    """RMS norm of a head [D]; w None: unchanged."""
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x) + eps) * np.asarray(w, dtype=np.float64)


def rotated(x, cos, sin, pair):
    """Rotation of the first 2*len(cos) values of a head [D]."""
    y = np.array(x, dtype=np.float64)
    h = len(cos)
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if pair else (i, i + h)
        y[a] = x[a] * cos[i] - x[b] * sin[i]
        y[b] = x[b] * cos[i] + x[a] * sin[i]
    return y


def attention(q, keys, values, n, scale):
    """One head: q [n, D], the last n of the len(keys) tokens.  Returns (out [n, D], the
    weighted sums of |values| [n, D], which bound what rounded weights can change)."""
    q, keys, values = (np.asarray(a, dtype=np.float64) for a in (q, keys, values))
    length, D = keys.shape
    out, mass = np.zeros((n, D)), np.zeros((n, D))
    for i in range(n):
        seen = length - n + i + 1
        if seen <= 0:
            continue
        s = scale * (keys[:seen] @ q[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        out[i], mass[i] = w @ values[:seen], w @ np.abs(values[:seen])
    return out, mass
