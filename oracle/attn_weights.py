"""Plain binary64 form of the accumulation of attention weights per cached row (test
infrastructure): one token at a time over the rows it sees, with bounds on what binary32
scores, logarithms and sums may be off by."""
from __future__ import annotations

import numpy as np

from oracle.attention import rows_of


def visible_rows(n_new, tokens_from, t, rows, table_row, block_size, num_pages, window, replay, base):
    """Rows token t of a request sees, and the slots that hold them."""
    pos = rows - n_new + (t - tokens_from)
    lo = max(0, pos - window + 1 if window else 0, replay)
    out = []
    for j in range(lo, pos + 1):
        logical = j // block_size - base
        if 0 <= logical < len(table_row) and 0 <= table_row[logical] < num_pages:
            out.append((j, int(table_row[logical]) * block_size + j % block_size))
    return out


def accumulate(q, lse, cache, qsl, seq_lens, table, block_size, rope_dim, scale, weights, decay=1.0, sink=None, window=0,
               replay=None, base=None, valid=None):
    """q binary64 [T, H, D]; returns (out, bound) with out NaN-free entries left as `weights`.

    Bounds, with u = 2^-23 for an operation on the tensor cores and 2^-24 elsewhere: a score is off by
    at most D u scale sum|q k| + 3 2^-24 |s|, the logarithm by 4 2^-24 |L| + 2^-23, exp2 by 2 ulp; a
    row's sum takes up to 128 plain additions in a row, the others being compensated; the result two
    more roundings."""
    T, H, D = q.shape
    out, tol = weights.astype(np.float64).copy(), np.zeros(weights.shape)
    for r in range(len(seq_lens)):
        rows, first, n = int(seq_lens[r]), int(qsl[r]), int(qsl[r + 1]) - int(qsl[r])
        end = min(rows, weights.shape[1])
        if end <= 0:
            continue
        total, off = np.zeros(end), np.zeros(end)
        for t in range(first, min(first + n, T)):
            if valid is not None and not valid[t]:
                continue
            seen = visible_rows(n, first, t, rows, table[r], block_size, cache.shape[0], window,
                                0 if replay is None else int(replay[r]), 0 if base is None else int(base[r]))
            seen = [(j, s) for j, s in seen if j < end]
            if not seen:
                continue
            at = [j for j, _ in seen]
            k = rows_of(cache, block_size, D, rope_dim, [s for _, s in seen])
            with np.errstate(all="ignore"):
                L = lse[t].astype(np.float64)
                if sink is not None:
                    L = np.logaddexp(L, sink.astype(np.float64))
                on = ~np.isneginf(L)
                if not on.any():
                    continue
                s = q[t][on] @ k.T * scale
                w = np.exp(s - L[on][:, None])
                rel = D * 2.0 ** -23 * scale * (np.abs(q[t][on]) @ np.abs(k).T) + 3 * 2.0 ** -24 * np.abs(s) \
                    + (4 * 2.0 ** -24 * np.abs(L[on]) + 2.0 ** -23)[:, None] + 2 * 2.0 ** -23
                # binary32 flushes what is below its range
                small = np.minimum(w, 2.0 ** -126)
                total[at] += w.sum(0)
                off[at] += (w * 1.01 * rel + small).sum(0)
        with np.errstate(all="ignore"):
            old = decay * weights[r, :end].astype(np.float64) if decay else np.zeros(end)
            out[r, :end] = old + total
            tol[r, :end] = off + total * 132 * 2.0 ** -24 + (np.abs(old) + total) * 2.0 ** -23
    return out, tol
