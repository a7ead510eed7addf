"""Plain Python forms of the batch-metadata steps (test infrastructure): one
request, token and page at a time, in Python integers."""
from __future__ import annotations

import numpy as np


def _slot(table, base, r, entry, block_size):
    if entry < 0:
        return -1
    logical = entry // block_size - (0 if base is None else int(base[r]))
    if not 0 <= logical < table.shape[1]:
        return -1
    page = int(table[r, logical])
    return -1 if page < 0 else page * block_size + entry % block_size


def compute_slot_mappings(qsl, seq_lens, table, block_size, num_tokens, base=None, comp_table=None,
                          comp_block_size=None, comp_base=None, ratio=1):
    """(positions, token_to_req, slots, compressed slots) of num_tokens tokens."""
    if comp_table is None:
        comp_table = table
    if comp_block_size is None:
        comp_block_size = block_size
    pos = np.full(num_tokens, -1, np.int64)
    req = np.full(num_tokens, -1, np.int32)
    slot = np.full(num_tokens, -1, np.int64)
    comp = np.full(num_tokens, -1, np.int64)
    for r in range(len(seq_lens)):
        first, end = int(qsl[r]), int(qsl[r + 1])
        for t in range(first, min(end, num_tokens)):
            p = int(seq_lens[r]) - (end - first) + (t - first)
            pos[t], req[t] = p, r
            slot[t] = _slot(table, base, r, p, block_size)
            if p >= 0 and (p + 1) % ratio == 0:
                comp[t] = _slot(comp_table, comp_base, r, p // ratio, comp_block_size)
    return pos, req, slot, comp


def extend_block_tables(seq_lens, pool, table, block_size, counts=None, head=0, ratio=1):
    """(table, counts, head, errors): the table grown row by row."""
    table = table.copy()
    width = table.shape[1]
    start = max(int(head), 0)
    head_out, errors = start, 0
    out = np.zeros(len(seq_lens), np.int32)
    for r, seq in enumerate(seq_lens):
        entries = max(int(seq), 0) // ratio
        need = -(-entries // block_size)
        have = 0 if counts is None else min(max(int(counts[r]), 0), width)
        more = 0 if need > width else max(need - have, 0)
        got = 0
        if start + more <= len(pool):
            got = more
            if more:
                head_out = start + more
        if need > width or (more > 0 and start + more > len(pool)):
            errors += 1
        for c in range(have, width):
            table[r, c] = pool[start + c - have] if c < have + got else -1
        out[r] = have + got
        start += more
    return table, out, head_out, errors
