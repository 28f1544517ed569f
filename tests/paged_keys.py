"""Attention over long contexts, checked key by key.

A tolerance for sums of that many random terms hides a key that was left out.  Two kinds of inputs do not:

counting   queries of 0: every key that a row sees has the same probability.  lse = ln(number of keys); V of a stage of
           16 keys is 1 in one feature and 0 in the others, so that out = (keys of the row with that feature) / (keys).
planted    K is 0 but for one key of each query row, aligned with it (a score of 39 or more above the others' 0): the
           row's output is that key's V, in every bit.
"""
from __future__ import annotations

import numpy as np

STAGE = 16


def features_of(table, feature, page_rows, head):
    """Feature of every stage of a request's pages: feature int [pages, kv_heads, page_rows / 16]."""
    return feature[np.asarray(table), head].reshape(-1)


def count_keys(stage_feature, seen, d, weight=None):
    """Keys of each feature among the first `seen` ones.  weight: how often each stage is counted (None: once)."""
    stages = -(-seen // STAGE)
    keys = np.full(stages, STAGE)
    keys[-1] = seen - (stages - 1) * STAGE
    if weight is not None:
        keys = keys * weight[:stages]
    return np.bincount(stage_feature[:stages], weights=keys, minlength=d)


def count_tols(counts, seen):
    """(out, lse) for counts [.., d] of rows that see `seen` [..] keys.

    All probabilities of a row are one number p = 2^-8 (the reference lies 8 above the score), taken to 2^-22 by ex2.  A
    lane adds at most two of them a stage to its sum (an uncut range: a quarter of the stages each; the other kernel one sum
    of a tile of 128 keys), then some 64 more follow: half a step of fp32 each.  bf16(p) is p's nearest, 2^-8, and counts
    times it are exact.  lse: the sum's logarithm to base 2 (up to 16) and the reference, 24 together: three roundings of
    half a step (2^-20) and one of log2f (2^-20).  out: bf16's half step besides."""
    seen = np.asarray(seen, np.float64)
    sums = 2.0 ** -22 + (seen / 32 + 64) * 2.0 ** -24
    v = counts / seen[..., None]
    return v * (2.0 ** -8 + 1.01 * sums[..., None] + 4 * 2.0 ** -24), sums + 4 * 2.0 ** -20


def count_errors(out, lse, counts, seen):
    """Largest errors of (out, lse) in units of what is allowed; out's zeros have to be zeros."""
    seen = np.asarray(seen, np.float64)
    tol, ltol = count_tols(counts, seen)
    want = counts / seen[..., None]
    off = np.abs(out - want)
    if not np.all(off[counts == 0] == 0):
        return np.inf, float(np.max(np.abs(lse - np.log(seen)) / ltol))
    return float(np.max(off[counts > 0] / tol[counts > 0])), float(np.max(np.abs(lse - np.log(seen)) / ltol))
