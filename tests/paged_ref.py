"""The paged cache in Python and numpy, 64 bits: the reference of the ff_paged_* tests.

The plan is the rule of the header taken literally, one request and one page after the other; attention
reads a request's rows from wherever the tables say they are.
"""
from __future__ import annotations

import math

import numpy as np

from tests.kv8_ref import lse_tol


class RefPaged:
    """Tables of a cache and the pools of one layer [pages, page_rows, kv_heads, d]."""

    def __init__(self, pages, page_rows, requests, capacity, kv_heads=1, d=1):
        self.pages, self.page_rows, self.requests, self.capacity = pages, page_rows, requests, capacity
        self.tables = np.zeros((requests, -(-capacity // page_rows)), np.int64)
        self.lengths = [0] * requests
        self.stack = list(range(pages - 1, -1, -1))  # the last element is the top
        self.first = [0] * (requests + 1)
        self.news = [0] * requests
        self.slots, self.positions = [], []
        self.dropped = False
        self.pool = {x: np.zeros((pages, page_rows, kv_heads, d)) for x in "kv"}

    def _pages(self, rows):
        return -(-rows // self.page_rows)

    def plan(self, n, counts, start=None):
        had = [self._pages(x) for x in self.lengths]
        kept = [x if start is None else min(max(int(s), 0), x) for x, s in zip(self.lengths, start or self.lengths)]
        self.dropped = False
        want, self.first = [], [0]
        for r in range(self.requests):
            c = min(max(int(counts[r]), 0), n)
            mine = min(c, n - self.first[-1])
            self.dropped |= mine < counts[r]
            self.first.append(self.first[-1] + mine)
            want.append(kept[r] + mine)
            if want[-1] > self.capacity:
                want[-1], self.dropped = self.capacity, True
        back = [int(self.tables[r, j]) for r in range(self.requests) for j in range(self._pages(want[r]), had[r])]
        self.stack += back[::-1]
        for r in range(self.requests):
            self.lengths[r] = want[r]
            for j in range(had[r], self._pages(want[r])):
                if not self.stack:
                    self.lengths[r] = j * self.page_rows
                    self.dropped = True
                    break
                self.tables[r, j] = self.stack.pop()
            self.news[r] = self.lengths[r] - kept[r]
        self.slots, self.positions = [-1] * n, [0] * n
        for r in range(self.requests):
            for i in range(self.news[r]):
                x = kept[r] + i
                self.slots[self.first[r] + i] = int(self.tables[r, x // self.page_rows]) * self.page_rows + x % self.page_rows
                self.positions[self.first[r] + i] = x

    def store(self, k, v):
        for i, slot in enumerate(self.slots[:len(k)]):
            if slot >= 0:
                self.pool["k"][slot // self.page_rows, slot % self.page_rows] = k[i]
                self.pool["v"][slot // self.page_rows, slot % self.page_rows] = v[i]

    def rows(self, x, r):
        """Rows that request r holds: [length, kv_heads, d]."""
        at = np.arange(self.lengths[r])
        return self.pool[x][self.tables[r, at // self.page_rows], at % self.page_rows]

    def attn(self, q, most=None):
        """(out, lse, tolerances of both), NaN where nothing is written."""
        n, heads, d = q.shape
        group = heads // self.pool["k"].shape[2]
        out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
        out_tol, ltol = np.zeros(q.shape), np.zeros(q.shape[:2])
        for r in range(self.requests):
            c, length, at = self.news[r], self.lengths[r], self.first[r]
            if c == 0 or (most is not None and c > most):
                continue
            take = max(0, min(c, n - at))
            k, v = self.rows("k", r), self.rows("v", r)
            seen = length - c + np.arange(take)[:, None] + 1
            hidden = np.arange(length) >= seen
            for h in range(heads):
                kh, vh = k[:, h // group], v[:, h // group]
                x = q[at:at + take, h]
                s = np.where(hidden, -np.inf, x @ kh.T / math.sqrt(d))
                top = s.max(1, keepdims=True)
                p = np.exp(s - top)
                z = p.sum(1, keepdims=True)
                o = p / z @ vh
                mag = np.where(hidden, 0.0, np.abs(x) @ np.abs(kh).T).max(1) / math.sqrt(d)
                out[at:at + take, h], lse[at:at + take, h] = o, (top + np.log(z))[:, 0]
                # bf16's half step of the result; of every probability its rounding (two bf16 pieces, 2^-16 at most, where
                # the call may meet up to 8 rows of a kv head; else one: bf16's half step, 2^-8), the scores' errors and
                # 2^-24 a key for the sums, relative to sum p |v|
                piece = 2.0 ** -16 if (n if most is None else most) * group <= 8 else 2.0 ** -8
                rel = piece + 2.0 * lse_tol(mag, d)[:, None] + length * 2.0 ** -24
                out_tol[at:at + take, h] = 2.0 ** -8 * np.abs(o) + 1.01 * rel * (p / z @ np.abs(vh))
                ltol[at:at + take, h] = lse_tol(mag, d) + length * 2.0 ** -24 + np.abs(lse[at:at + take, h]) * 2.0 ** -24
        return out, lse, out_tol, ltol
