"""Beam search's selection: the best continuations over beams and vocabulary, in fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).
"""
from __future__ import annotations

import numpy as np

LOWEST = -2.0 ** 125          # logits up to here are no candidates and add nothing to a sum


def sum_against_largest(x):
    """(largest, log(sum(exp(x - largest)))) of one row; NaN where the row has no candidates."""
    x = np.asarray(x, np.float64)
    x = np.where(x <= LOWEST, -np.inf, x)
    if np.any(np.isnan(x)) or np.any(x > -LOWEST) or not np.any(x > -np.inf):
        return np.nan, np.nan
    top = x.max()
    return float(top), float(np.log(np.exp(x - top).sum()))


def log_sum(x) -> float:
    """log(sum(exp(x))) of one row; NaN where the row has no candidates."""
    return float(sum(sum_against_largest(x)))


def select(logits, scores, n, finished=None, end_token=0):
    """logits [B, K, V], scores [B, K] -> (scores [B, n] fp64, parents, tokens, finished [B, n],
    gap [B]): gap is the smallest difference between neighbouring scores of different beams
    among the first n + 1 candidates."""
    logits, scores = np.asarray(logits, np.float64), np.asarray(scores, np.float64)
    B, K, V = logits.shape
    out = (np.full((B, n), -np.inf), np.full((B, n), -1, np.int64), np.full((B, n), -1, np.int64),
           np.zeros((B, n), bool))
    gap = np.full(B, np.inf)
    for b in range(B):
        cand = []                                            # (score, beam, rank in the beam, token)
        for k in range(K):
            s = scores[b, k]
            if not np.isfinite(s):
                continue
            if finished is not None and finished[b, k]:
                cand.append((s, k, 0, end_token))
                continue
            top, total = sum_against_largest(logits[b, k])
            if np.isnan(total):
                continue
            row = logits[b, k]
            order = np.lexsort((np.arange(V), -row))[: n + 1]
            cand += [(s + ((row[v] - top) - total), k, i, int(v)) for i, v in enumerate(order) if row[v] > LOWEST]
        cand.sort(key=lambda c: (-c[0], c[1], c[2]))
        for i, (s, k, _, v) in enumerate(cand[:n]):
            out[0][b, i], out[1][b, i], out[2][b, i] = s, b * K + k, v
            out[3][b, i] = finished is not None and (bool(finished[b, k]) or v == end_token)
        for a, c in zip(cand[:n], cand[1:n + 1]):
            if a[1] != c[1]:
                gap[b] = min(gap[b], a[0] - c[0])
    return (*out, gap)
