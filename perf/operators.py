"""Workloads of the attention and page-table operators: what each computes, its inputs and the sizes it is used at.

Four kinds of case:

* ``sparse``  attention of new tokens over the rows of paged fp8_ds_mla caches that an index matrix names: window
              columns in the sliding-window cache, top-k columns in the compressed cache (sparse_mla_attention);
* ``chunk``   causal attention of a chunk of new tokens over the positions of their own requests through the block
              table, over the whole context or a sliding window (chunk_mla_attention);
* ``slots``   positions, token-to-request map and cache slots of a batch from its request lengths
              (compute_slot_mappings);
* ``tables``  block tables grown from request lengths and a list of unused pages (extend_block_tables).

``run`` computes them from elementary torch operations, or through ``paged_sparse_kv_gb300.ops`` where ``own`` is set;
``exact`` computes the same values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---- sizes ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of one request with the heads of one rank of a tensor-parallel group: latency alone
        _sparse("sparse one token", tokens=1, heads=16, window=128, topk=512, context=8192),
        # the decode batch: 64 requests x 1 token, window 128, top-k 512
        _sparse("sparse decode", tokens=64, heads=64, window=128, topk=512, context=8192),
        # the decode part of a mixed batch: top-k 1024, an odd number of tokens, 128 heads
        _sparse("sparse mixed", tokens=317, heads=128, window=128, topk=1024, context=32768),
        # odd sizes: 24 heads, a 256-dim record, pages of 16, a top-k that fills no tile
        _sparse("sparse odd", tokens=97, heads=24, window=37, topk=163, context=3000, head_dim=256, block=16),
        # a prefill chunk of 4096 new tokens from position 0: the first rows have few entries
        _sparse("sparse prefill", tokens=4096, heads=128, window=128, topk=512, context=4096, prefill=True),
        # a layer without compressed entries, decode: the window alone
        _chunk("chunk window decode", reqs=64, tokens=64, heads=64, window=128, context=8192),
        # a ragged chunk of new tokens over long prefixes, the heads of one rank, full causal
        _chunk("chunk ragged", reqs=3, tokens=1901, heads=16, window=0, context=6144),
        # single tokens over a long context: the work is split along the keys
        _chunk("chunk long context", reqs=2, tokens=2, heads=64, window=0, context=131072),
        # the decode batch's metadata: one token per request
        _slots("slots decode", reqs=256, tokens=256, context=32768, ratio=4),
        # the metadata of a large ragged prefill batch
        _slots("slots prefill", reqs=37, tokens=1000003, context=131072, ratio=4),
        # decode growth: few requests cross a page border
        _tables("tables decode", reqs=256, context=8192, held=True),
        # block tables of many long requests from nothing
        _tables("tables long", reqs=2048, context=131072, held=False),
    ]


def _sparse(name, tokens, heads, window, topk, context, head_dim=512, rope=64, block=64, prefill=False):
    return {"name": name, "kind": "sparse", "tokens": tokens, "heads": heads, "window": window, "topk": topk,
            "context": context, "head_dim": head_dim, "rope": rope, "block": block, "prefill": prefill}


def _chunk(name, reqs, tokens, heads, window, context, head_dim=512, rope=64, block=64):
    return {"name": name, "kind": "chunk", "reqs": reqs, "tokens": tokens, "heads": heads, "window": window,
            "context": context, "head_dim": head_dim, "rope": rope, "block": block}


def _slots(name, reqs, tokens, context, ratio, block=64):
    return {"name": name, "kind": "slots", "reqs": reqs, "tokens": tokens, "context": context, "ratio": ratio,
            "block": block}


def _tables(name, reqs, context, held, block=64, ratio=1):
    return {"name": name, "kind": "tables", "reqs": reqs, "context": context, "held": held, "block": block,
            "ratio": ratio}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["sparse", "sparse", "chunk", "chunk", "slots", "tables"])
    if kind in ("sparse", "chunk"):
        heads = rng.choice([8, 16, 32, 64, 128, rng.randint(1, 128)])
        head_dim = rng.choice([512, 512, 256, 128])
        rope = rng.choice([64, 64, 0])
        block = rng.choice([64, 64, 16, 32])
    if kind == "sparse":
        prefill = rng.random() < 0.3
        tokens = _log(rng, 64, 4096) if prefill else _log(rng, 1, 512)
        c = _sparse(None, tokens, heads, rng.choice([128, rng.randint(1, 256)]),
                    rng.choice([512, 1024, rng.randint(1, 2048)]), tokens if prefill else _log(rng, 1024, 32768),
                    head_dim, rope, block, prefill)
        while _keys_sparse(c) * c["heads"] > 4096 * 128 * 500:
            c["tokens"] = max(1, c["tokens"] // 2)
    elif kind == "chunk":
        if rng.random() < 0.5:
            reqs = _log(rng, 1, 128)
            tokens, window, context = reqs, rng.choice([0, 128, rng.randint(1, 1024)]), _log(rng, 512, 32768)
        else:
            reqs = rng.randint(1, 5)
            tokens = reqs + _log(rng, 16, 2048)
            window, context = rng.choice([0, 128, rng.randint(1, 2048)]), tokens + _log(rng, 16, 4096)
        c = _chunk(None, reqs, tokens, heads, window, context, head_dim, rope, block)
        while _keys_chunk(c) * c["heads"] > 1901 * 16 * 5000 or c["reqs"] * c["context"] > 1 << 20:
            c["heads"] = max(1, c["heads"] // 2)
            c["context"] = max(c["tokens"] + 16, c["context"] // 2)
            if c["heads"] == 1 and c["context"] == c["tokens"] + 16:
                c["tokens"] = max(c["reqs"], c["tokens"] // 2)
    elif kind == "slots":
        reqs = _log(rng, 1, 1024)
        tokens = reqs + _log(rng, 1, 1 << 19)
        c = _slots(None, reqs, tokens, tokens + _log(rng, 64, 65536), rng.choice([1, 4, 128]), rng.choice([64, 16, 48]))
    else:
        c = _tables(None, _log(rng, 1, 2048), _log(rng, 64, 65536), rng.random() < 0.5, rng.choice([64, 16, 48]),
                    rng.choice([1, 4]))
    del c["name"]
    return c


# ---- lengths: fixed by the case, so that its work is known ---------------------------------------------------------

def _lens_rng(case):
    """A generator that depends on the case's own sizes alone (not on the seed)."""
    sizes = [int(v) for k, v in sorted(case.items()) if k not in ("name", "kind")]
    return np.random.default_rng([20261206] + sizes)


def _entries_sparse(case):
    """(window entries, top-k entries) of each token, and its position."""
    T, W, K = case["tokens"], case["window"], case["topk"]
    if case["prefill"]:
        pos = np.arange(T, dtype=np.int64)
    else:
        lo = max(1, case["context"] // 8)
        pos = _lens_rng(case).integers(lo, case["context"] + 1, size=T).astype(np.int64) - 1
    nw = np.minimum(W, pos + 1)
    # about 5% of a full decode row is trailing -1
    nk = np.minimum(K if case["prefill"] else K - K // 20, (pos + 1) // 4)
    return nw, nk, pos


def _keys_sparse(case):
    nw, nk, _ = _entries_sparse(case)
    return int((nw + nk).sum())


def _query_lens(case):
    """Query length and context (prefix + query) of each request: every request has at least one new token."""
    R, T = case["reqs"], case["tokens"]
    rng = _lens_rng(case)
    if T == R:
        q = np.ones(R, dtype=np.int64)
    else:
        cut = np.sort(rng.choice(np.arange(1, T), size=R - 1, replace=False)) if R > 1 else np.zeros(0, dtype=np.int64)
        q = np.diff(np.concatenate([[0], cut, [T]])).astype(np.int64)
    room = np.maximum(case["context"] - q, 0)
    seq = q + (room * rng.uniform(0.125, 1.0, size=R)).astype(np.int64)
    if case["kind"] == "chunk" and R == T and case["context"] >= 65536:
        seq[:] = case["context"] - np.arange(R)  # long contexts of nearly one length
    return q, seq


def _keys_chunk(case):
    q, seq = _query_lens(case)
    total = 0
    for n, s in zip(q, seq):
        pos = np.arange(s - n, s)
        total += int(np.minimum(pos + 1, case["window"] or 1 << 40).sum())
    return total


def _table_lens(case):
    rng = _lens_rng(case)
    seq = rng.integers(max(1, case["context"] // 8), case["context"] + 1, size=case["reqs"]).astype(np.int64)
    # tokens the rows of the table already hold pages for: all but the newest one, or none
    before = seq - 1 if case["held"] else np.zeros_like(seq)
    pages = lambda n: -(-(n // case["ratio"]) // case["block"])  # noqa: E731
    return seq, pages(before), pages(seq)


# ---- inputs -------------------------------------------------------------------------------------------------------

def _page_stride(case):
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    return -(-bs * (D + rope + D // 64) // 16) * 16


def _cache(case, pages, gen):
    """A cache of `pages` fp8_ds_mla pages holding N(0, 1) rows, quantised with a power-of-two scale per 64 dims."""
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    nope, slots = D - rope, pages * bs
    cache = torch.zeros((pages, _page_stride(case)), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (D * bs))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n * bs, D), generator=gen, device=DEV).to(torch.bfloat16)
        b = x[:, :nope].float().reshape(n * bs, nope // 64, 64)
        e = torch.ceil(torch.log2(b.abs().amax(2).clamp_min(1e-4) / 448.0))
        codes = (b * torch.exp2(-e)[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        row = torch.cat([codes.reshape(n * bs, nope), x[:, nope:].contiguous().view(torch.uint8).reshape(n * bs, 2 * rope)], 1)
        scales = torch.zeros((n * bs, D // 64), dtype=torch.uint8, device=DEV)
        scales[:, :nope // 64] = (e + 127.0).to(torch.uint8)
        cache[p:p + n, :bs * (D + rope)] = row.reshape(n, -1)
        cache[p:p + n, bs * (D + rope):bs * (D + rope + D // 64)] = scales.reshape(n, -1)
    assert slots <= 2**31 - 1
    return cache


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    st = {"case": dict(case)}
    if case["kind"] in ("sparse", "chunk"):
        T, H, D = case["tokens"], case["heads"], case["head_dim"]
        st["q"] = (torch.randn((T, H, D), generator=gen, device=DEV) * 2.0).to(torch.bfloat16)
        st["scale"] = D ** -0.5
        st["sink"] = torch.randn((H,), generator=gen, device=DEV)
    if case["kind"] == "sparse":
        bs, W, K = case["block"], case["window"], case["topk"]
        nw, nk, pos = _entries_sparse(case)
        # the window cache holds the last positions of each request, the compressed one an entry for four positions
        per_w = -(-(int(pos.max()) + 1 if case["prefill"] else W + bs) // bs)
        per_k = max(1, -(-((int(pos.max()) + 1) // 4) // bs))
        reqs = 1 if case["prefill"] else case["tokens"]
        pages_w, pages_k = reqs * per_w, min(reqs * per_k, max(per_k, 65536 // bs))
        st["cache"], st["extra"] = _cache(case, pages_w, gen), _cache(case, pages_k, gen)
        table_w = torch.randperm(pages_w, generator=gen, device=DEV).reshape(reqs, per_w)
        table_k = torch.stack([torch.randperm(pages_k, generator=gen, device=DEV)[:per_k] for _ in range(min(reqs, 64))])
        req = torch.zeros(len(pos), dtype=torch.int64, device=DEV) if case["prefill"] else torch.arange(len(pos), device=DEV)
        p = torch.from_numpy(pos).to(DEV)[:, None]
        n_w, n_k = (torch.from_numpy(n).to(DEV)[:, None] for n in (nw, nk))
        c = torch.arange(W, device=DEV)[None, :]
        w = (p - n_w + 1 + c) % (per_w * bs)
        w = torch.where(c < n_w, table_w[req[:, None], w // bs] * bs + w % bs, -1)
        # distinct compressed entries below (pos + 1) // 4: a stride that is odd against a power of two above the range
        c = torch.arange(K, device=DEV)[None, :]
        n = ((p + 1) // 4).clamp_min(1)
        start = torch.randint(0, 1 << 30, (len(pos), 1), generator=gen, device=DEV) % n
        k = (start + c * (n // n_k.clamp_min(1)).clamp_min(1)) % n
        k = torch.where(c < n_k, table_k[req[:, None] % table_k.shape[0], k // bs] * bs + k % bs, -1)
        pad = torch.full((len(pos), -K % 4), -1, dtype=torch.int64, device=DEV)
        st["indices"] = torch.cat([w, k, pad], 1).to(torch.int32)
    elif case["kind"] == "chunk":
        q, seq = _query_lens(case)
        bs, R = case["block"], case["reqs"]
        width = -(-int(seq.max()) // bs)
        pages = -(-seq // bs)
        perm = rng.permutation(int(pages.sum()))
        table = np.full((R, width), -1, dtype=np.int32)
        at = 0
        for r in range(R):
            table[r, :pages[r]] = perm[at:at + pages[r]]
            at += pages[r]
        st["cache"] = _cache(case, int(pages.sum()), gen)
        st["qsl"], st["seq"] = _i32(np.concatenate([[0], np.cumsum(q)])), _i32(seq)
        st["t2r"], st["table"] = _i32(np.repeat(np.arange(R), q)), _i32(table)
        st["most_q"], st["most_s"] = int(q.max()), int(seq.max())
    elif case["kind"] == "slots":
        q, seq = _query_lens(case)
        bs, R = case["block"], case["reqs"]
        st["qsl"], st["seq"] = _i32(np.concatenate([[0], np.cumsum(q)])), _i32(seq)
        wide = lambda n: -(-n // bs)  # noqa: E731
        st["table"] = torch.randint(0, 1 << 20, (R, wide(int(seq.max()))), generator=gen, device=DEV).to(torch.int32)
        st["ctable"] = torch.randint(0, 1 << 20, (R, max(1, wide(int(seq.max()) // case["ratio"]))), generator=gen, device=DEV).to(torch.int32)
    else:
        seq, held, need = _table_lens(case)
        total, width = int(held.sum()), max(1, int(need.max()))
        spare = int((need - held).sum()) + 5
        pool = torch.randperm(total + spare, generator=gen, device=DEV).to(torch.int32)
        table = np.full((case["reqs"], width), -1, dtype=np.int32)
        perm = pool[:total].cpu().numpy()
        at = 0
        for r in np.nonzero(held)[0]:
            table[r, :held[r]] = perm[at:at + held[r]]
            at += held[r]
        st["seq"], st["held"], st["table"] = _i32(seq), _i32(held), _i32(table)
        st["pool"], st["head"] = pool, _i32([total])
    return st


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"sparse": _plain_sparse, "chunk": _plain_chunk, "slots": _plain_slots, "tables": _plain_tables}[st["case"]["kind"]](st)


def _run_own(st):
    from paged_sparse_kv_gb300 import ops
    c = st["case"]
    if c["kind"] == "sparse":
        return ops.sparse_mla_attention(st["q"], st["cache"], st["indices"], c["block"], extra_cache=st["extra"],
                                        extra_block_size=c["block"], split=c["window"], softmax_scale=st["scale"],
                                        sink=st["sink"], rope_dim=c["rope"])
    if c["kind"] == "chunk":
        return ops.chunk_mla_attention(st["q"], st["cache"], st["qsl"], st["seq"], st["t2r"], st["table"], c["block"],
                                       window_size=c["window"], softmax_scale=st["scale"], sink=st["sink"],
                                       rope_dim=c["rope"])
    if c["kind"] == "slots":
        return ops.compute_slot_mappings(st["qsl"], st["seq"], st["table"], c["block"], c["tokens"],
                                         compressed_block_table=st["ctable"], compressed_block_size=c["block"],
                                         compress_ratio=c["ratio"])
    return ops.extend_block_tables(st["seq"], st["pool"], st["table"], c["block"], page_counts=st["held"],
                                   pool_head=st["head"], compress_ratio=c["ratio"])


def _plain_rows(cache, case, slots):
    """The rows of `slots` (any shape, each inside the cache) in binary32."""
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    nope, ts = D - rope, D + rope
    data = cache[:, :bs * ts].unflatten(1, (bs, ts))
    scales = cache[:, bs * ts:bs * (ts + D // 64)].unflatten(1, (bs, D // 64))
    page, off = slots // bs, slots % bs
    row = data[page, off]
    scale = torch.exp2(scales[page, off][..., :nope // 64].float() - 127.0)
    x = row[..., :nope].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (nope // 64, 64)) * scale[..., None]
    x = x.flatten(-2)
    return torch.cat([x, row[..., nope:].contiguous().view(torch.bfloat16).float()], -1) if rope else x


def _plain_softmax(s, visible, sink):
    """Weights of the visible entries (last dim), with the sink's share of the sum, and log of the sum without it."""
    s = torch.where(visible, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / (total + torch.exp(sink - top))
    return p, (torch.log(total) + top).squeeze(-1)


def _plain_sparse(st):
    c, idx = st["case"], st["indices"].long()
    W, bs = c["window"], c["block"]
    room = torch.full((idx.shape[1],), st["extra"].shape[0] * bs, device=idx.device)
    room[:W] = st["cache"].shape[0] * bs
    visible = (idx >= 0) & (idx < room)
    slots = torch.where(visible, idx, 0)
    k = torch.cat([_plain_rows(st["cache"], c, slots[:, :W]), _plain_rows(st["extra"], c, slots[:, W:])], 1)
    k = torch.where(visible[..., None], k, 0.0)
    s = torch.bmm(st["q"].float(), k.transpose(1, 2)) * st["scale"]
    p, lse = _plain_softmax(s, visible[:, None, :], st["sink"][None, :, None])
    return torch.bmm(p, k).to(torch.bfloat16), lse


def _plain_chunk(st):
    c = st["case"]
    R, H, D, bs, Q, L = c["reqs"], c["heads"], c["head_dim"], c["block"], st["most_q"], st["most_s"]
    t2r, qsl, seq = st["t2r"].long(), st["qsl"].long(), st["seq"].long()
    t = torch.arange(c["tokens"], device=DEV)
    n = qsl[1:] - qsl[:-1]
    pos = seq[t2r] - n[t2r] + t - qsl[t2r]
    at = t2r * Q + t - qsl[t2r]  # the token's row among Q rows of its request
    q = torch.zeros((R * Q, H, D), device=DEV)
    q[at] = st["q"].float()
    place = torch.full((R * Q,), -1, dtype=torch.int64, device=DEV)
    place[at] = pos
    key = torch.arange(L, device=DEV)
    page = st["table"].long()[:, key // bs]
    k = _plain_rows(st["cache"], c, torch.where(page >= 0, page * bs + key % bs, 0))
    k = torch.where((page >= 0)[..., None], k, 0.0)
    place = place.reshape(R, Q, 1, 1)
    visible = (key <= place) & (key > place - (c["window"] or L + 1)) & (page >= 0)[:, None, None, :]
    s = torch.bmm(q.reshape(R, Q * H, D), k.transpose(1, 2)).reshape(R, Q, H, L) * st["scale"]
    p, lse = _plain_softmax(s, visible, st["sink"][None, None, :, None])
    o = torch.bmm(p.reshape(R, Q * H, L), k).reshape(R * Q, H, D)
    return o[at].to(torch.bfloat16), lse.reshape(R * Q, H)[at]


def _plain_slots(st):
    c, qsl, seq = st["case"], st["qsl"].long(), st["seq"].long()
    t = torch.arange(c["tokens"], device=DEV)
    r = torch.bucketize(t, qsl, right=True) - 1
    pos = seq[r] - (qsl[r + 1] - qsl[r]) + t - qsl[r]
    bs, ratio = c["block"], c["ratio"]
    slot = st["table"].long()[r, pos // bs] * bs + pos % bs
    e = pos // ratio
    page = st["ctable"].long()[r, (e // bs).clamp_max(st["ctable"].shape[1] - 1)]
    closes = (pos + 1) % ratio == 0
    return pos, r.to(torch.int32), slot, torch.where(closes, page * bs + e % bs, -1)


def _plain_tables(st):
    c, table = st["case"], st["table"]
    held = st["held"].long()
    entries = st["seq"].long() // c["ratio"]
    need = torch.maximum((entries + c["block"] - 1) // c["block"], held)
    more = need - held
    first = st["head"].long() + torch.cumsum(more, 0) - more
    col = torch.arange(table.shape[1], device=DEV)
    at = first[:, None] + col - held[:, None]
    new = (col >= held[:, None]) & (col < need[:, None])
    grown = torch.where(new, st["pool"][torch.where(new, at, 0)], torch.where(col < held[:, None], table, -1))
    return grown, need.to(torch.int32), (st["head"].long() + more.sum()).to(torch.int32)


# ---- what a pass cannot do without -------------------------------------------------------------------------------------

def work(case):
    if case["kind"] in ("sparse", "chunk"):
        T, H, D = case["tokens"], case["heads"], case["head_dim"]
        record = D + case["rope"] + D // 64
        io = T * H * D * 2 * 2 + T * H * 4 + H * 4
        if case["kind"] == "sparse":
            nw, nk, pos = _entries_sparse(case)
            keys = int((nw + nk).sum())
            if case["prefill"]:
                rows = int(pos.max()) + 1 + int(nk.max() and (pos.max() + 1) // 4)
            else:
                rows = min(keys, int(nw.sum()) + 65536)
            return {"bytes": io + rows * record + T * (case["window"] + -(-case["topk"] // 4) * 4) * 4, "flops": 4 * keys * H * D}
        q, seq = _query_lens(case)
        lo = np.maximum(seq - q - (case["window"] or 1 << 40) + 1, 0)
        pages = int((-(-seq // case["block"])).sum())
        return {"bytes": io + int((seq - lo).sum()) * record + pages * 4 + T * 4, "flops": 4 * _keys_chunk(case) * H * D}
    if case["kind"] == "slots":
        q, seq = _query_lens(case)
        touched = int((q // case["block"] + 1).sum()) + int((q // case["ratio"] // case["block"] + 1).sum())
        return {"bytes": case["tokens"] * (8 + 4 + 8 + 8) + case["reqs"] * 8 + touched * 4, "flops": 0}
    seq, held, need = _table_lens(case)
    more = int((need - held).sum())
    # the new entries are read from the pool; every entry past the held ones is written
    return {"bytes": more * 4 + 4 * int((max(1, int(need.max())) - held).sum()) + case["reqs"] * 12, "flops": 0}


# ---- the same in 64 bits ------------------------------------------------------------------------------------------------

def _e4m3_values():
    """The value of each E4M3 byte: sign, 4 exponent bits with bias 7, 3 mantissa bits; no infinities."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = math.nan if b & 127 == 127 else (-x if b & 128 else x)
    return torch.from_numpy(v)


def _exact_rows(cache, case, slots):
    """[n, D] rows in binary64 of a flat list of slots, byte by byte from the flat cache."""
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    nope = D - rope
    flat = cache.reshape(-1)
    base = (slots // bs) * cache.shape[1]
    at = base + (slots % bs) * (nope + 2 * rope)
    codes = flat[at[:, None] + torch.arange(nope, device=DEV)].long()
    out = torch.empty((len(slots), D), dtype=torch.float64, device=DEV)
    sc = flat[(base + bs * (nope + 2 * rope) + (slots % bs) * (D // 64))[:, None] + torch.arange(nope // 64, device=DEV)]
    out[:, :nope] = _e4m3_values().to(DEV)[codes] * torch.pow(2.0, sc.double() - 127.0).repeat_interleave(64, 1)
    for j in range(rope):  # a bf16 value is the upper half of a binary32
        b = flat[(at + nope + 2 * j)[:, None] + torch.arange(2, device=DEV)].int()
        out[:, nope + j] = ((b[:, 0] << 16) | (b[:, 1] << 24)).view(torch.float32).double()
    return out


def _exact_attend(q, k, mask, scale, sink):
    """One set of keys [n, D] for query rows [..., D] under a mask [..., n]: softmax with a sink, and the log of the sum."""
    s = (q @ k.T) * scale
    s = s.masked_fill(~mask, -math.inf)
    top = torch.maximum(s.amax(-1), sink)
    e = torch.exp(s - top[..., None])
    n = e.sum(-1)
    return (e @ k) / (n + torch.exp(sink - top))[..., None], torch.log(n) + top


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "sparse":
        T, H, D, W, bs = case["tokens"], case["heads"], case["head_dim"], case["window"], case["block"]
        out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
        lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
        rows = [_exact_rows(c, case, torch.arange(c.shape[0] * bs, device=DEV)) for c in (st["cache"], st["extra"])]
        idx = st["indices"].long()
        for t in range(T):
            keys = []
            for part, r in ((idx[t, :W], rows[0]), (idx[t, W:], rows[1])):
                keys.append(r[part.clamp(0, len(r) - 1)])
            seen = torch.cat([(idx[t, :W] >= 0) & (idx[t, :W] < len(rows[0])), (idx[t, W:] >= 0) & (idx[t, W:] < len(rows[1]))])
            out[t], lse[t] = _exact_attend(st["q"][t].double(), torch.cat(keys), seen[None, :], st["scale"], st["sink"].double())
        return out, lse
    if case["kind"] == "chunk":
        q, seq = _query_lens(case)
        T, H, D, bs = case["tokens"], case["heads"], case["head_dim"], case["block"]
        out = torch.zeros((T, H, D), dtype=torch.float64, device=DEV)
        lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
        t = 0
        for r in range(case["reqs"]):
            p = torch.arange(int(seq[r]), device=DEV)
            k = _exact_rows(st["cache"], case, st["table"][r].long()[p // bs] * bs + p % bs)
            for first in range(0, int(q[r]), 128):
                n = min(128, int(q[r]) - first)
                pos = int(seq[r] - q[r]) + first + torch.arange(n, device=DEV)
                mask = (p[None, :] <= pos[:, None]) & (p[None, :] > pos[:, None] - (case["window"] or 1 << 40))
                out[t:t + n], lse[t:t + n] = _exact_attend(st["q"][t:t + n].double(), k, mask[:, None, :].expand(n, H, len(p)),
                                                           st["scale"], st["sink"].double()[None, :])
                t += n
        return out, lse
    host = {k: v.cpu().numpy().astype(np.int64) for k, v in st.items() if isinstance(v, torch.Tensor)}
    if case["kind"] == "slots":
        bs, ratio = case["block"], case["ratio"]
        pos, req, slot, comp = (np.empty(case["tokens"], dtype=np.int64) for _ in range(4))
        for r in range(case["reqs"]):
            a, b = host["qsl"][r], host["qsl"][r + 1]
            p = np.arange(host["seq"][r] - (b - a), host["seq"][r])
            pages = lambda n, row: row[n // bs] * bs + n % bs  # noqa: E731
            pos[a:b], req[a:b], slot[a:b] = p, r, pages(p, host["table"][r])
            last = (p + 1) % ratio == 0  # the token that completes its group of `ratio`
            comp[a:b] = -1
            comp[a:b][last] = pages(p[last] // ratio, host["ctable"][r])
        return pos, req.astype(np.int32), slot, comp
    table, at, counts = host["table"].copy(), int(host["head"][0]), []
    for r in range(case["reqs"]):
        n, have = -(-(int(host["seq"][r]) // case["ratio"]) // case["block"]), int(host["held"][r])
        table[r, have:] = -1
        if n > have:
            table[r, have:n] = host["pool"][at:at + n - have]
            at += n - have
        counts.append(max(n, have))
    return table.astype(np.int32), np.array(counts, dtype=np.int32), np.array([at], dtype=np.int32)
