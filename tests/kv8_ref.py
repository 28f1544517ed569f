"""The 8-bit cache in numpy, 64 bits: the reference of the ff_kv8_* tests.

A sequence's cache is a list of blocks per kv head; values are kept as (code value, scale exponent)
so that what a store rounds is rounded here by the definition (nearest e4m3 number, ties to even),
not by a conversion instruction.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64
E_MIN, E_MAX = -96, 112


def nearest8(x: np.ndarray) -> np.ndarray:
    """x rounded to the nearest e4m3 number, ties to even, saturating at 448; NaN stays NaN."""
    x = np.clip(np.asarray(x, np.float64), -448.0, 448.0)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.round(x / step) * step


def exponent(values: np.ndarray) -> int:
    """Smallest e with the largest finite magnitude <= 448 * 2^e, within the bounds."""
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    top = float(v.max()) if v.size else 0.0
    if top == 0.0:
        return E_MIN
    m, e = math.frexp(top)            # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return max(E_MIN, min(E_MAX, e - 9 if m <= 0.875 else e - 8))


class RefCache:
    """One layer: codes [batch, rows, kv_heads, d] (as numbers) and scale exponents [batch, blocks, kv_heads]."""

    def __init__(self, batch, capacity, kv_heads, d):
        self.capacity, self.blocks = capacity, -(-capacity // BLOCK)
        rows = self.blocks * BLOCK
        self.code = {x: np.zeros((batch, rows, kv_heads, d)) for x in "kv"}
        self.e = {x: np.full((batch, self.blocks, kv_heads), E_MIN) for x in "kv"}
        self.length = np.zeros(batch, np.int64)
        self.batch, self.kv_heads, self.d = batch, kv_heads, d

    def _write(self, x, b, t, h, r0, stay, values):
        """Rows r0 .. of block t take `values`; the `stay` rows before them stay."""
        e = exponent(values)
        base = t * BLOCK
        if stay:
            e = max(e, int(self.e[x][b, t, h]))
            old = self.code[x][b, base:base + stay, h]
            self.code[x][b, base:base + stay, h] = nearest8(np.ldexp(old, int(self.e[x][b, t, h]) - e))
        self.code[x][b, base + r0:base + r0 + len(values), h] = nearest8(np.ldexp(values, -e))
        self.e[x][b, t, h] = e

    def append(self, k, v, start=None, counts=None):
        n = k.shape[1]
        for b in range(self.batch):
            held = int(self.length[b])
            s = held if start is None else min(max(int(start[b]), 0), held)
            c = n if counts is None else min(max(int(counts[b]), 0), n)
            c = min(c, self.capacity - s)
            for t in range(s // BLOCK, -(-(s + c) // BLOCK) if c else 0):
                lo, hi = max(s, t * BLOCK), min(s + c, (t + 1) * BLOCK)
                for x, new in (("k", k), ("v", v)):
                    for h in range(self.kv_heads):
                        self._write(x, b, t, h, lo - t * BLOCK, lo - t * BLOCK, new[b, lo - s:hi - s, h])
            self.length[b] = s + c

    def values(self, x, b, h, n=None):
        n = int(self.length[b]) if n is None else n
        return np.ldexp(self.code[x][b, :n, h], np.repeat(self.e[x][b, :, h], BLOCK)[:n, None])

    def load(self, n, start=None):
        got = {x: np.zeros((self.batch, n, self.kv_heads, self.d)) for x in "kv"}
        for b in range(self.batch):
            s = 0 if start is None else int(start[b])
            lo, hi = max(s, 0), min(s + n, int(self.length[b]))
            if hi > lo:
                for x in "kv":
                    for h in range(self.kv_heads):
                        got[x][b, lo - s:hi - s, h] = self.values(x, b, h)[lo:hi]
        return got["k"], got["v"]

    def attn(self, q, causal=False, counts=None, weights=None):
        """(out, lse, weights, tolerances): NaN in out and lse where nothing is written."""
        batch, n, heads, d = q.shape
        group = heads // self.kv_heads
        out = np.full(q.shape, np.nan)
        lse = np.full(q.shape[:3], np.nan)
        spread = np.zeros(q.shape)          # sum p |v|
        mag = np.zeros(q.shape[:3])         # largest sum |q| |k| / sqrt(d) over the keys seen
        w = None if weights is None else np.array(weights, np.float64)
        wtol = None if weights is None else np.zeros_like(w)
        for b in range(batch):
            length = int(self.length[b])
            c = n if counts is None else min(max(int(counts[b]), 0), n)
            for h in range(self.kv_heads):
                k, v = self.values("k", b, h), self.values("v", b, h)
                for g in range(h * group, (h + 1) * group):
                    for i in range(c):
                        seen = max(0, length - c + i + 1) if causal else length
                        if not seen:
                            out[b, i, g], lse[b, i, g] = 0.0, -np.inf
                            continue
                        s = k[:seen] @ q[b, i, g] / math.sqrt(d)
                        top = s.max()
                        p = np.exp(s - top)
                        z = p.sum()
                        lse[b, i, g] = top + math.log(z)
                        p /= z
                        out[b, i, g] = p @ v[:seen]
                        spread[b, i, g] = p @ np.abs(v[:seen])
                        m = (np.abs(k[:seen]) @ np.abs(q[b, i, g])).max() / math.sqrt(d)
                        mag[b, i, g] = m
                        if w is not None:
                            w[b, h, :seen] += p
                            wtol[b, h, :seen] += p * (2 * lse_tol(m, d) + heads * n * 2.0 ** -23)
        return out, lse, w, (spread, mag, wtol)

    def evict(self, weights, n_keep, n_recent, dst):
        """(kept, weights_out); fills dst."""
        kept = np.full((self.batch, self.kv_heads, n_keep), -1, np.int64)
        wout = np.zeros((self.batch, self.kv_heads, dst.capacity))
        for b in range(self.batch):
            length = int(self.length[b])
            count = min(length, n_keep)
            for h in range(self.kv_heads):
                w = np.asarray(weights[b, h, :length], np.float64)
                if length <= n_keep:
                    rows = np.arange(length)
                else:
                    old = length - n_recent
                    key = np.where(np.isnan(w[:old]), -np.inf, w[:old])
                    nan = np.isnan(w[:old])
                    order = sorted(range(old), key=lambda j: (nan[j], -key[j], j))
                    rows = np.array(sorted(order[:n_keep - n_recent]) + list(range(old, length)), np.int64)
                kept[b, h, :count] = rows
                wout[b, h, :count] = w[rows]
                for x in "kv":
                    vals = self.values(x, b, h)[rows]
                    for t in range(-(-count // BLOCK)):
                        dst._write(x, b, t, h, 0, 0, vals[t * BLOCK:(t + 1) * BLOCK])
            dst.length[b] = count
        return kept, wout


def lse_tol(mag, d):
    """Error of a score and of the log-sum: the products of two f16 numbers are exact in fp32, their sum of d takes at
    most d roundings (allowed: truncation, 2^-23 of the running sum, which is at most mag); the factor and the K
    scale one each; then 2^x and the logarithm, 2^-22 relative each, and the fp32 value of the result itself."""
    return (d + 8) * 2.0 ** -23 * mag + 2.0 ** -20


def out_tol(out, spread, mag, d, n_keys):
    """bf16's half step of the result; f16's half step of every probability (2^-11), the error of the scores in the
    probabilities, and 2^-24 a key for the sums, all relative to sum p |v|; probabilities below f16's normal range are
    off by at most 2^-25 of 2^-8, relative to the row's largest."""
    rel = 2.0 ** -11 + 2.0 * lse_tol(mag, d)[..., None] + n_keys * 2.0 ** -24
    return 2.0 ** -8 * np.abs(out) + 1.01 * rel * spread
