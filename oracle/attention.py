"""Plain binary64 form of attention over paged fp8_ds_mla caches (test
infrastructure): one token at a time over the rows the C oracle's gather gives,
with bounds on how far binary32 sums and one bf16 rounding of the weights and
of the result may be from it."""
from __future__ import annotations

import numpy as np

import oracle


def bf16_bits_to_f64(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rows_of(cache, block_size, head_dim, rope_dim, slots):
    """Binary64 rows of int slots (each inside the cache)."""
    idx = np.asarray(slots, np.int32).reshape(1, -1)
    if idx.size == 0:
        return np.zeros((0, head_dim))
    return bf16_bits_to_f64(oracle.dequantize_and_gather_k_cache(cache, block_size, 0, head_dim,
                                                                 rope_dim, idx)[0])


def attend(q, k, scale, sink):
    """One token: q [H, D] and visible rows k [n, D] in binary64.  Returns out
    [H, D], lse [H] and the bounds of both.

    Bounds, with u = 2^-23 for an operation on the tensor cores (which need not
    round to nearest) and 2^-24 elsewhere: a score is off by at most
    ds = D u scale sum|q k| + 3 2^-24 |s|, so a weight and the sum of the weights
    by a factor within exp(+-ds), to which exp2's own error (2 ulp), its argument
    reduction (|s - m| 2^-23) and n additions of the sum add; each weight is
    rounded to bf16 once (2^-8 of it) and the weighted sum takes n additions;
    the result is rounded to bf16 (2^-8 of it)."""
    H, D = q.shape
    n = k.shape[0]
    if n == 0:
        z = np.zeros((H, D))
        return z, np.full(H, -np.inf), z, np.zeros(H)
    u = 2.0 ** -23
    with np.errstate(all="ignore"):
        s = q @ k.T * scale
        m = s.max(1)
        e = np.exp(s - m[:, None])
        total = e.sum(1)
        den = total + (0.0 if sink is None else np.exp(sink - m))
        out = (e @ k) / den[:, None]
        lse = m + np.log(total)
        ds = D * u * scale * (np.abs(q) @ np.abs(k).T).max(1) + 3 * u * np.abs(s).max(1)
        rel = 2 * (ds + 2 * u + u * (m - s.min(1)).clip(0, 200) + n * u)
        mass = (e @ np.abs(k)) / den[:, None]
        tol = mass * (2.0 ** -8 + rel[:, None] + n * u) * 1.01 + np.abs(out) * 2.0 ** -8 * 1.01 + 1e-37
        tol_lse = rel + 4 * u + np.abs(lse) * u
    return out, lse, tol, tol_lse


def sparse_mla_attention(q, cache, indices, block_size, rope_dim, scale, sink=None, extra=None,
                         extra_block_size=None, split=None):
    """q binary64 [T, H, D]; caches uint8; returns (out, lse, bound, lse bound)."""
    T, H, D = q.shape
    C = indices.shape[1]
    split = C if split is None else split
    res = [np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H, D)), np.zeros((T, H))]
    for t in range(T):
        rows = []
        for c, bs, part in ((cache, block_size, indices[t, :split]),
                            (extra, extra_block_size, indices[t, split:])):
            if part.size:
                part = part[(part >= 0) & (part < c.shape[0] * bs)]
                rows.append(rows_of(c, bs, D, rope_dim, part))
        k = np.concatenate(rows) if rows else np.zeros((0, D))
        for dst, v in zip(res, attend(q[t], k, scale, sink)):
            dst[t] = v
    return res


def visible_slots(t, qsl, seq_lens, t2r, table, block_size, num_pages, window, replay=None, base=None,
                  valid=None):
    r = int(t2r[t])
    if not 0 <= r < len(seq_lens) or (valid is not None and not valid[t]):
        return np.zeros(0, np.int64)
    pos = int(seq_lens[r]) - int(qsl[r + 1] - qsl[r]) + (t - int(qsl[r]))
    lo = max(0, pos - window + 1 if window else 0, 0 if replay is None else int(replay[r]))
    slots = []
    for p in range(lo, pos + 1):
        logical = p // block_size - (0 if base is None else int(base[r]))
        if 0 <= logical < table.shape[1] and 0 <= table[r, logical] < num_pages:
            slots.append(int(table[r, logical]) * block_size + p % block_size)
    return np.array(slots, np.int64)


def chunk_mla_attention(q, cache, qsl, seq_lens, t2r, table, block_size, rope_dim, scale, sink=None,
                        window=0, replay=None, base=None, valid=None):
    T, H, D = q.shape
    res = [np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H, D)), np.zeros((T, H))]
    for t in range(T):
        s = visible_slots(t, qsl, seq_lens, t2r, table, block_size, cache.shape[0], window, replay,
                          base, valid)
        k = rows_of(cache, block_size, D, rope_dim, s)
        for dst, v in zip(res, attend(q[t], k, scale, sink)):
            dst[t] = v
    return res
