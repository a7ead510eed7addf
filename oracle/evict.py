"""Plain Python forms of eviction from a cache (test infrastructure): one request and
one row at a time."""
from __future__ import annotations

import math

import numpy as np


def select(weights, seq_lens, keep_lens, positions=None, first=0, recent=0):
    """(list of moves, new length, weights and positions afterwards, error) per request."""
    res = []
    for r, n in enumerate(int(x) for x in seq_lens):
        if n > weights.shape[1]:
            res.append(([], n, None, None, True))
            continue
        n = max(n, 0)
        m = min(n, max(int(keep_lens[r]), 0))
        w = [float(x) for x in weights[r, :n]]
        p = list(range(n)) if positions is None else [int(x) for x in positions[r, :n]]
        newest = max(p, default=0)

        def rank(j):  # smaller comes first
            safe = p[j] < first or (recent > 0 and p[j] > newest - recent)
            return (0 if safe else 1, 0.0 if safe or math.isnan(w[j]) else -w[j], j) if safe or not math.isnan(w[j]) \
                else (2, 0.0, j)
        kept = set(sorted(range(n), key=rank)[:m])
        moves = list(zip([j for j in range(m, n) if j in kept], [j for j in range(m) if j not in kept]))
        rows = list(range(m))
        for a, b in moves:
            rows[b] = a
        res.append((moves, m, [weights[r, j] for j in rows], [p[j] for j in rows], False))
    return res


def move(cache, block_size, data, scale, table, moves, num_moves, base=None):
    """(cache afterwards, moves not made)."""
    cache, errors = cache.copy(), 0
    for r in range(len(num_moves)):
        for src, dst in moves[r][:max(0, min(int(num_moves[r]), len(moves[r])))]:
            at = []
            for row in (int(src), int(dst)):
                logical = row // block_size - (0 if base is None else int(base[r]))
                page = int(table[r, logical]) if row >= 0 and 0 <= logical < table.shape[1] else -1
                at.append((page, row % block_size) if 0 <= page < cache.shape[0] else None)
            if None in at:
                errors += 1
                continue
            (a, i), (b, j) = at
            cache[b, j * data:(j + 1) * data] = cache[a, i * data:(i + 1) * data]
            o = block_size * data
            cache[b, o + j * scale:o + (j + 1) * scale] = cache[a, o + i * scale:o + (i + 1) * scale]
    return cache, errors
