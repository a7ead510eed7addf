"""Workloads of rotary positions and of eviction from a bounded cache: what each computes, its inputs and the sizes it is used at.

Four kinds of case:

* ``table``    cosines and sines of positions, unscaled or scaled for long contexts (build_rope_cos_sin_cache);
* ``rotary``   the rotation of a part of each head of queries and keys, interleaved or half layout, forward or inverse
               (apply_rotary_embedding);
* ``weights``  attention weights summed per cached row over new tokens and heads, added to decayed earlier ones
               (accumulate_attention_weights);
* ``evict``    the rows a cache keeps by their weights, and the records moved to where the others were
               (select_cache_evictions and move_cache_rows).

``run`` computes them from elementary torch operations, or through ``paged_sparse_kv_gb300.ops`` where ``own`` is set;
``exact`` computes the same values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- sizes ------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the table of a model served at its trained length
        _table("table trained length", positions=8192, dim=64, theta=10000.0),
        # the table of a context extended sixteenfold, by parts
        _table("table extended", positions=1 << 20, dim=64, theta=160000.0, scaling="yarn", factor=16.0, original=65536),
        # the decode batch: 64 tokens, the rope dims of 64 heads and of the new key rows
        _rotary("rotary decode", tokens=64, heads=64, keys=1, head_dim=512, offset=448, rope=64, part=True),
        # a prefill chunk of 4096 tokens, 128 heads
        _rotary("rotary prefill", tokens=4096, heads=128, keys=1, head_dim=512, offset=448, rope=64, part=True),
        # odd sizes, half layout, whole heads of which a part in front is turned back
        _rotary("rotary odd inverse", tokens=1901, heads=33, keys=3, head_dim=256, offset=0, rope=96, half=True, inverse=True),
        # one new token of one request: latency alone
        _weights("weights one token", reqs=1, tokens=1, heads=16, context=8192),
        # the decode batch: 64 requests x 1 token
        _weights("weights decode", reqs=64, tokens=64, heads=64, context=8192),
        # the last tokens of long prompts score all rows: ragged, 40 heads, pages of 16, earlier weights fading
        _weights("weights last tokens", reqs=5, tokens=203, heads=40, context=31000, block=16, decay=0.97),
        # every token of a prefill chunk
        _weights("weights prefill", reqs=1, tokens=4096, heads=128, context=4096),
        # a decode step at the bound: one row more than the budget in each of 64 requests
        _evict("evict one row", reqs=64, context=2049, keep=2048, full=True),
        # prompts compressed after prefill
        _evict("evict prompts", reqs=16, context=32768, keep=4096, full=False),
        # few long requests, odd sizes, indexer keys
        _evict("evict long odd", reqs=3, context=131071, keep=50001, full=False, record="mxfp4", block=48),
    ]


def _table(name, positions, dim, theta, scaling="none", factor=1.0, original=0):
    return {"name": name, "kind": "table", "positions": positions, "dim": dim, "theta": theta, "scaling": scaling,
            "factor": factor, "original": original}


def _rotary(name, tokens, heads, keys, head_dim, offset, rope, part=False, half=False, inverse=False, dtype="bf16"):
    """part: the rotated dims alone are taken out of the heads, as a view of them, into tensors of their own."""
    return {"name": name, "kind": "rotary", "tokens": tokens, "heads": heads, "keys": keys, "head_dim": head_dim,
            "offset": offset, "rope": rope, "part": part, "half": half, "inverse": inverse, "dtype": dtype}


def _weights(name, reqs, tokens, heads, context, window=0, head_dim=512, rope=64, block=64, decay=1.0):
    return {"name": name, "kind": "weights", "reqs": reqs, "tokens": tokens, "heads": heads, "context": context,
            "window": window, "head_dim": head_dim, "rope": rope, "block": block, "decay": decay}


def _evict(name, reqs, context, keep, full, record="fp8", block=64, first=4, recent=64):
    return {"name": name, "kind": "evict", "reqs": reqs, "context": context, "keep": keep, "full": full, "record": record,
            "block": block, "first": first, "recent": recent}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["table", "rotary", "rotary", "weights", "weights", "weights", "evict", "evict"])
    if kind == "table":
        scaling = rng.choice(["none", "linear", "yarn"])
        dim = rng.choice([64, 64, 128, 32, 2 * rng.randint(1, 128)])
        c = _table(None, min(_log(rng, 512, 1 << 20), (1 << 26) // dim), dim, rng.choice([10000.0, 160000.0, 500000.0]), scaling,
                   1.0 if scaling == "none" else rng.choice([4.0, 16.0, rng.uniform(1.5, 40.0)]),
                   rng.choice([4096, 8192, 65536]) if scaling == "yarn" else 0)
    elif kind == "rotary":
        heads, keys = rng.choice([8, 16, 64, 128, rng.randint(1, 128)]), rng.choice([1, 1, rng.randint(1, 8)])
        head_dim = rng.choice([512, 256, 128, 64, 2 * rng.randint(16, 256)])
        rope = rng.choice([min(64, head_dim), head_dim, 2 * rng.randint(1, head_dim // 2)])
        c = _rotary(None, _log(rng, 1, 8192), heads, keys, head_dim, rng.choice([0, head_dim - rope, rng.randint(0, head_dim - rope)]),
                    rope, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.4, rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[c["dtype"]]
        while c["tokens"] * (heads + keys) * head_dim * size > 1 << 29:
            c["tokens"] = max(1, c["tokens"] // 2)
    elif kind == "weights":
        heads = rng.choice([8, 16, 32, 64, 128, rng.randint(1, 128)])
        head_dim, rope, block = rng.choice([512, 512, 256, 128]), rng.choice([64, 64, 0]), rng.choice([64, 64, 16, 32])
        window, decay = rng.choice([0, 0, rng.randint(1, 4096)]), rng.choice([1.0, 1.0, 0.0, rng.uniform(0.5, 1.0)])
        if rng.random() < 0.5:
            reqs = _log(rng, 1, 128)
            tokens, context = reqs, _log(rng, 512, 32768)
        else:
            reqs = rng.randint(1, 5)
            tokens = reqs + _log(rng, 16, 2048)
            context = tokens + _log(rng, 16, 16384)
        c = _weights(None, reqs, tokens, heads, context, window, head_dim, rope, block, decay)
        while _pairs(c) * c["heads"] * head_dim > 2048 * 4096 * 128 * 512 or c["reqs"] * c["context"] > 1 << 20:
            c["heads"] = max(1, c["heads"] // 2)
            c["context"] = max(c["tokens"] + 16, c["context"] // 2)
            if c["heads"] == 1 and c["context"] == c["tokens"] + 16:
                c["tokens"] = max(c["reqs"], c["tokens"] // 2)
    else:
        reqs, context = _log(rng, 1, 128), _log(rng, 64, 131072)
        while reqs * context > 1 << 19:
            reqs, context = max(1, reqs // 2), (context // 2 if reqs == 1 else context)
        keep = rng.choice([context - 1, context // 8, rng.randint(1, context)])
        c = _evict(None, reqs, context, max(1, keep), rng.random() < 0.5, rng.choice(["fp8", "fp8", "mxfp4", "fp8_indexer"]),
                   rng.choice([64, 64, 16, 48]), rng.choice([0, 4, 16]), rng.choice([0, 32, 256]))
    del c["name"]
    return c


# ---- lengths: fixed by the case, so that its work is known ---------------------------------------------------------

def _lens_rng(case):
    """A generator that depends on the case's own sizes alone (not on the seed)."""
    sizes = [int(v) for k, v in sorted(case.items()) if k in ("reqs", "tokens", "heads", "context", "keep", "block", "window")]
    return np.random.default_rng([20261208] + sizes)


def _query_lens(case):
    """New tokens and cached rows (theirs included) of each request: every request has at least one new token."""
    R, T = case["reqs"], case["tokens"]
    rng = _lens_rng(case)
    if T == R:
        q = np.ones(R, dtype=np.int64)
    else:
        cut = np.sort(rng.choice(np.arange(1, T), size=R - 1, replace=False)) if R > 1 else np.zeros(0, dtype=np.int64)
        q = np.diff(np.concatenate([[0], cut, [T]])).astype(np.int64)
    room = np.maximum(case["context"] - q, 0)
    seq = q + (room * rng.uniform(0.125, 1.0, size=R)).astype(np.int64)
    if R == 1:
        seq[:] = max(case["context"], T)
    return q, seq


def _pairs(case):
    """(token, row) pairs the masks leave."""
    q, seq = _query_lens(case)
    total = 0
    for n, s in zip(q, seq):
        pos = np.arange(s - n, s)
        total += int(np.minimum(pos + 1, case["window"] or 1 << 40).sum())
    return total


def _evict_lens(case):
    if case["full"]:
        return np.full(case["reqs"], case["context"], dtype=np.int64)
    return _lens_rng(case).integers(max(1, case["context"] // 2), case["context"] + 1, size=case["reqs"]).astype(np.int64)


# ---- inputs -------------------------------------------------------------------------------------------------------

def _page_stride(case):
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    return -(-bs * (D + rope + D // 64) // 16) * 16


def _cache(case, pages, gen):
    """A cache of `pages` fp8_ds_mla pages holding N(0, 1) rows, quantised with a power-of-two scale per 64 dims."""
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    nope = D - rope
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
    return cache


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _block_table(rng, lens, bs):
    """Each request's pages, in a random order of all pages; -1 past them."""
    pages = -(-lens // bs)
    perm = rng.permutation(int(pages.sum()))
    table = np.full((len(lens), int(pages.max())), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, at


EVICT_DIMS = {"fp8": (512, 576, 8), "mxfp4": (128, 64, 4), "fp8_indexer": (128, 128, 4)}  # head_dim, data bytes, scale bytes


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    st = {"case": dict(case), "seed": seed}
    if case["kind"] == "table":
        # where the table starts: a program that serves many contexts builds it in pieces
        st["first"] = int(rng.integers(0, 1 << 16))
    elif case["kind"] == "rotary":
        T, D, rope = case["tokens"], case["head_dim"], case["rope"]
        dt, most = DTYPES[case["dtype"]], 32768
        st["q"] = torch.randn((T, case["heads"], D), generator=gen, device=DEV).to(dt)
        st["k"] = torch.randn((T, case["keys"], D), generator=gen, device=DEV).to(dt)
        st["positions"] = torch.randint(0, most, (T,), generator=gen, device=DEV)
        f = 10000.0 ** (-2.0 * torch.arange(rope // 2, device=DEV, dtype=torch.float64) / rope)
        a = torch.arange(most, device=DEV, dtype=torch.float64)[:, None] * f
        st["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        if case["part"]:
            cut = slice(case["offset"], case["offset"] + rope)
            st["q"], st["k"] = st["q"][..., cut], st["k"][..., cut]
        st["offset"] = 0 if case["part"] else case["offset"]
    elif case["kind"] == "weights":
        T, H, D, bs = case["tokens"], case["heads"], case["head_dim"], case["block"]
        q, seq = _query_lens(case)
        table, pages = _block_table(rng, seq, bs)
        st["q"] = (torch.randn((T, H, D), generator=gen, device=DEV) * 2.0).to(torch.bfloat16)
        st["cache"] = _cache(case, pages, gen)
        st["scale"] = D ** -0.5
        st["sink"] = torch.randn((H,), generator=gen, device=DEV)
        st["qsl"], st["seq"], st["table"] = _i32(np.concatenate([[0], np.cumsum(q)])), _i32(seq), _i32(table)
        st["weights"] = torch.rand((case["reqs"], int(seq.max())), generator=gen, device=DEV)
        st["out"] = torch.zeros_like(st["weights"])
        # the attention's log of the sum, of these queries over these rows
        st["lse"] = torch.empty((T, H), device=DEV)
        for r, first, n, rows, t0, t1 in _pieces(case):
            s = _scores(st, r, first, rows, t0, t1)
            st["lse"][first + t0:first + t1] = torch.logsumexp(s, -1)
        del st["rows"], st["rows_of"]
    else:
        D, data, scale = EVICT_DIMS[case["record"]]
        lens, bs = _evict_lens(case), case["block"]
        table, pages = _block_table(rng, lens, bs)
        width = int(lens.max())
        st["cache"] = torch.randint(0, 256, (pages, -(-bs * (data + scale) // 16) * 16), generator=gen, device=DEV, dtype=torch.uint8)
        st["table"], st["lens"] = _i32(table), _i32(lens)
        st["keep"] = _i32(np.full(case["reqs"], case["keep"]))
        # accumulated weights: a few rows hold most of it, many nothing that binary32 sees
        w = torch.exp(torch.randn((case["reqs"], width), generator=gen, device=DEV) * 3.0)
        st["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=DEV) < 0.1, 0.0, w)
        # positions of rows that earlier evictions have left out of order and with gaps
        p = torch.cumsum(torch.randint(1, 4, w.shape, generator=gen, device=DEV), 1)
        st["positions"] = torch.gather(p, 1, torch.argsort(p + torch.randint(0, 512, p.shape, generator=gen, device=DEV), 1)).to(torch.int32)
        st["weights_out"], st["positions_out"] = torch.zeros_like(w), torch.zeros_like(st["positions"])
        st["moves"] = torch.full((case["reqs"], width // 2, 2), -1, dtype=torch.int32, device=DEV)
    return st


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"table": _plain_table, "rotary": _plain_rotary, "weights": _plain_weights, "evict": _plain_evict}[st["case"]["kind"]](st)


def _run_own(st):
    from paged_sparse_kv_gb300 import ops
    c = st["case"]
    if c["kind"] == "table":
        return ops.build_rope_cos_sin_cache(c["positions"], c["dim"], theta=c["theta"], scaling=c["scaling"], factor=c["factor"],
                                            original_positions=c["original"], first_position=st["first"], device=DEV)
    if c["kind"] == "rotary":
        return ops.apply_rotary_embedding(st["positions"], st["q"], st["cos_sin"], st["k"], rope_offset=st["offset"],
                                          interleaved=not c["half"], inverse=c["inverse"])
    if c["kind"] == "weights":
        return ops.accumulate_attention_weights(st["q"], st["lse"], st["cache"], st["qsl"], st["seq"], st["table"], c["block"],
                                                st["weights"], decay=c["decay"], window_size=c["window"],
                                                softmax_scale=st["scale"], sink=st["sink"], rope_dim=c["rope"], out=st["out"])
    moves, counts, lens, w, p = ops.select_cache_evictions(st["weights"], st["lens"], st["keep"], row_positions=st["positions"],
                                                           num_first=c["first"], num_recent=c["recent"],
                                                           weights_out=st["weights_out"], positions_out=st["positions_out"],
                                                           moves=st["moves"])
    record = {"fp8": ops.PSK_REC_FP8_DS_MLA, "mxfp4": ops.PSK_REC_MXFP4, "fp8_indexer": ops.PSK_REC_FP8_INDEXER}[c["record"]]
    ops.move_cache_rows(st["cache"], st["table"], moves, counts, c["block"], EVICT_DIMS[c["record"]][0], record=record)
    return moves, counts, lens, w, p, st["cache"]


def _frequencies(c):
    """Radians per position of each pair, in 64 bits."""
    i = torch.arange(c["dim"] // 2, device=DEV, dtype=torch.float64)
    f = c["theta"] ** (-2.0 * i / c["dim"])
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "yarn":
        # pairs that turn more than 32 times over the original length keep their frequency, those that turn less
        # than once are stretched, and a ramp joins them
        pair = lambda turns: c["dim"] * math.log(c["original"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(c["theta"]))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), c["dim"] - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * keep + f / c["factor"] * (1.0 - keep)
    return f


def _plain_table(st):
    c = st["case"]
    p = torch.arange(st["first"], st["first"] + c["positions"], device=DEV, dtype=torch.float64)
    a = p[:, None] * _frequencies(c)
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _plain_rotary(st):
    c, o, n = st["case"], st["offset"], st["case"]["rope"] // 2
    cs = st["cos_sin"][st["positions"]][:, None, :]
    cos, sin = cs[..., :n], (-cs[..., n:] if c["inverse"] else cs[..., n:])
    out = []
    for x in (st["q"], st["k"]):
        y = x.clone(memory_format=torch.contiguous_format)
        part = x[..., o:o + 2 * n].float()
        a, b = (part[..., :n], part[..., n:]) if c["half"] else (part[..., 0::2], part[..., 1::2])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        y[..., o:o + 2 * n] = (torch.cat([ra, rb], -1) if c["half"] else torch.stack([ra, rb], -1).flatten(-2)).to(x.dtype)
        out.append(y)
    return tuple(out)


def _plain_rows(st, r, rows):
    """The first `rows` rows of a request in binary32."""
    c = st["case"]
    D, rope, bs = c["head_dim"], c["rope"], c["block"]
    nope, ts, cache = D - rope, D + rope, st["cache"]
    page = st["table"][r, :-(-rows // bs)].long()
    data = cache[page][:, :bs * ts].reshape(-1, ts)[:rows]
    scale = torch.exp2(cache[page][:, bs * ts:bs * (ts + D // 64)].reshape(-1, D // 64)[:rows, :nope // 64].float() - 127.0)
    x = data[:, :nope].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (nope // 64, 64)) * scale[..., None]
    return torch.cat([x.flatten(-2), data[:, nope:].contiguous().view(torch.bfloat16).float()], 1)


def _pieces(case):
    """(request, its first token, its tokens, its rows, a range of its tokens) of at most 2^28 scores at a time."""
    q, seq = _query_lens(case)
    first = 0
    for r in range(case["reqs"]):
        step = max(1, (1 << 28) // (case["heads"] * int(seq[r])))
        for t0 in range(0, int(q[r]), step):
            yield r, first, int(q[r]), int(seq[r]), t0, min(int(q[r]), t0 + step)
        first += int(q[r])


def _scores(st, r, first, rows, t0, t1):
    """[tokens, heads, rows] scores of tokens t0 .. t1 of a request, -infinity where they see nothing."""
    c = st["case"]
    n = int(_query_lens(c)[0][r])
    if st.get("rows_of") != r:
        st["rows_of"], st["rows"] = r, _plain_rows(st, r, rows)
    s = (st["q"][first + t0:first + t1].float() @ st["rows"].T) * st["scale"]
    j = torch.arange(rows, device=DEV)
    pos = (rows - n + torch.arange(t0, t1, device=DEV))[:, None]
    seen = (j <= pos) & (j > pos - (c["window"] or 1 << 30))
    return torch.where(seen[:, None, :], s, -math.inf)


def _plain_weights(st):
    c = st["case"]
    lse = torch.logaddexp(st["lse"], st["sink"])
    out, at = st["out"], -1
    st.pop("rows_of", None)
    for r, first, n, rows, t0, t1 in _pieces(c):
        if r != at:
            at, total = r, torch.zeros(rows, dtype=torch.float64, device=DEV)
        e = torch.exp(_scores(st, r, first, rows, t0, t1) - lse[first + t0:first + t1, :, None])
        total += e.sum(1).double().sum(0)
        if t1 == n:
            out[r, :rows] = (c["decay"] * st["weights"][r, :rows].double() + total).float()
    return out


def _plain_evict(st):
    c, w, p = st["case"], st["weights"], st["positions"]
    R, width = w.shape
    n, j = st["lens"].long()[:, None], torch.arange(width, device=DEV)[None, :]
    m = torch.minimum(n, st["keep"].long()[:, None])
    there = j < n
    newest = torch.where(there, p, -1).amax(1, keepdim=True)
    safe = (p < c["first"]) | (p > newest - c["recent"])
    key = torch.where(there, torch.where(safe, math.inf, w.double()), -math.inf)
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, j.expand(R, width))
    kept = there & (rank < m)
    hole, mover = ~kept & (j < m), kept & (j >= m)
    counts = hole.sum(1)
    moves = st["moves"]
    for col, flag in ((0, mover), (1, hole)):
        r, i = torch.nonzero(flag, as_tuple=True)
        moves[r, (torch.cumsum(flag, 1) - 1)[r, i], col] = i.to(torch.int32)
    live = torch.arange(moves.shape[1], device=DEV)[None, :] < counts[:, None]
    r, i = torch.nonzero(live, as_tuple=True)
    src, dst = moves[r, i, 0].long(), moves[r, i, 1].long()
    for x, y in ((w, st["weights_out"]), (p, st["positions_out"])):
        y.copy_(torch.where(j < m, x, y))
        y[r, dst] = x[r, src]
    _, data, scale = EVICT_DIMS[c["record"]]
    bs, table = c["block"], st["table"].long()
    rows = st["cache"][:, :bs * data].unflatten(1, (bs, data))
    scales = st["cache"][:, bs * data:bs * (data + scale)].unflatten(1, (bs, scale))
    for x in (rows, scales):
        x[table[r, dst // bs], dst % bs] = x[table[r, src // bs], src % bs]
    return moves, counts.to(torch.int32), m[:, 0].to(torch.int32), st["weights_out"], st["positions_out"], st["cache"]


# ---- what a pass cannot do without -------------------------------------------------------------------------------------

def work(case):
    if case["kind"] == "table":
        n = case["positions"] * case["dim"]
        return {"bytes": 4 * n, "flops": 5 * n}
    if case["kind"] == "rotary":
        T, rows = case["tokens"], case["tokens"] * (case["heads"] + case["keys"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * rows * (case["rope"] if case["part"] else case["head_dim"]) * size + T * (8 + 4 * case["rope"]),
                "flops": 3 * rows * case["rope"]}
    if case["kind"] == "weights":
        T, H, D = case["tokens"], case["heads"], case["head_dim"]
        q, seq = _query_lens(case)
        lo = np.maximum(seq - q - (case["window"] or 1 << 40) + 1, 0)
        old = 4 if case["decay"] else 0
        return {"bytes": T * H * (2 * D + 4) + H * 4 + int((seq - lo).sum()) * (D + case["rope"] + D // 64)
                + int(seq.sum()) * (4 + old) + int((-(-seq // case["block"])).sum()) * 4,
                "flops": 2 * _pairs(case) * H * (D + 2)}
    lens = _evict_lens(case)
    m = np.minimum(lens, case["keep"])
    _, data, scale = EVICT_DIMS[case["record"]]
    # a row past the new length is kept, and moved, as often as one before it
    moves = int((m * (lens - m) / np.maximum(lens, 1)).sum())
    return {"bytes": int(lens.sum()) * 8 + int(m.sum()) * 8 + moves * (8 + 2 * (data + scale)), "flops": 0}


# ---- the same in 64 bits ------------------------------------------------------------------------------------------------

def _e4m3_values():
    """The value of each E4M3 byte: sign, 4 exponent bits with bias 7, 3 mantissa bits; no infinities."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = math.nan if b & 127 == 127 else (-x if b & 128 else x)
    return torch.from_numpy(v)


def _exact_rows(st, case, r, rows):
    """[rows, D] in binary64, byte by byte from the flat cache."""
    D, rope, bs = case["head_dim"], case["rope"], case["block"]
    nope, cache = D - rope, st["cache"]
    flat, j = cache.reshape(-1), torch.arange(rows, device=DEV)
    base = st["table"][r].long()[j // bs] * cache.shape[1]
    at = base + (j % bs) * (nope + 2 * rope)
    out = torch.empty((rows, D), dtype=torch.float64, device=DEV)
    codes = flat[at[:, None] + torch.arange(nope, device=DEV)].long()
    sc = flat[(base + bs * (nope + 2 * rope) + (j % bs) * (D // 64))[:, None] + torch.arange(nope // 64, device=DEV)]
    out[:, :nope] = _e4m3_values().to(DEV)[codes] * torch.pow(2.0, sc.double() - 127.0).repeat_interleave(64, 1)
    for i in range(rope):  # a bf16 value is the upper half of a binary32
        b = flat[(at + nope + 2 * i)[:, None] + torch.arange(2, device=DEV)].int()
        out[:, nope + i] = ((b[:, 0] << 16) | (b[:, 1] << 24)).view(torch.float32).double()
    return out


def _exact_table(case, st):
    d, out = case["dim"], torch.empty((case["positions"], case["dim"]), dtype=torch.float64, device=DEV)
    for i in range(d // 2):
        f = math.exp(-2.0 * i / d * math.log(case["theta"]))
        if case["scaling"] == "linear":
            f /= case["factor"]
        elif case["scaling"] == "yarn":
            at = [d / 2 * math.log(case["original"] / (2 * math.pi * b), case["theta"]) for b in (32.0, 1.0)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
            ramp = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            f *= 1.0 - ramp + ramp / case["factor"]
        a = torch.arange(case["positions"], device=DEV, dtype=torch.float64).add_(st["first"]).mul_(f)
        out[:, i], out[:, d // 2 + i] = a.cos(), a.sin()
    return out


def _exact_rotary(case, st):
    res = []
    n, o = case["rope"] // 2, st["offset"]
    cs = st["cos_sin"].double()[st["positions"]]
    turn = torch.complex(cs[:, :n], cs[:, n:])
    if case["inverse"]:
        turn = turn.conj()
    for x in (st["q"].double(), st["k"].double()):
        y = x.clone()
        first, second = (slice(o, o + n), slice(o + n, o + 2 * n)) if case["half"] else (slice(o, o + 2 * n, 2), slice(o + 1, o + 2 * n, 2))
        v = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
        y[..., first], y[..., second] = v.real, v.imag
        res.append(y)
    return tuple(res)


def _exact_weights(case, st):
    q, seq = _query_lens(case)
    out = st["out"].double()
    first = 0
    for r in range(case["reqs"]):
        n, rows = int(q[r]), int(seq[r])
        k = _exact_rows(st, case, r, rows)
        total = torch.zeros(rows, dtype=torch.float64, device=DEV)
        j = torch.arange(rows, device=DEV)
        step = max(1, (1 << 27) // (rows * case["heads"]))
        for a in range(0, n, step):
            b = min(n, a + step)
            pos = rows - n + torch.arange(a, b, device=DEV)[:, None, None]
            lse = st["lse"][first + a:first + b].double()
            den = torch.exp(lse) + torch.exp(st["sink"].double())  # these sums are far from the range's ends
            e = torch.exp(st["q"][first + a:first + b].double() @ k.T * st["scale"]) / den[..., None]
            e = e.masked_fill((j > pos) | (j <= pos - (case["window"] or 1 << 40)), 0.0)
            total += e.sum((0, 1))
        out[r, :rows] = case["decay"] * st["weights"][r, :rows].double() + total
        first += n
    return out


def _exact_evict(case, st):
    host = {k: v.cpu().numpy() for k, v in st.items() if isinstance(v, torch.Tensor) and k != "cache"}
    moves, w_out, p_out = host["moves"].copy(), host["weights_out"].astype(np.float64), host["positions_out"].copy()
    cache, lens, counts = st["cache"].clone(), [], []
    _, data, scale = EVICT_DIMS[case["record"]]
    bs = case["block"]
    for r in range(case["reqs"]):
        n = int(host["lens"][r])
        m = min(n, int(host["keep"][r]))
        w, p = host["weights"][r, :n].astype(np.float64), host["positions"][r, :n]
        w = np.where((p < case["first"]) | (p > p.max() - case["recent"]), np.inf, w)
        kept = np.zeros(n, dtype=bool)
        kept[np.lexsort((np.arange(n), -w))[:m]] = True
        dst, src = np.flatnonzero(~kept[:m]), m + np.flatnonzero(kept[m:])
        moves[r, :len(dst), 0], moves[r, :len(dst), 1] = src, dst
        for x, y in ((host["weights"], w_out), (host["positions"], p_out)):
            y[r, :m] = x[r, :m]
            y[r, dst] = x[r, src]
        page = lambda i: torch.from_numpy(host["table"][r, i // bs].astype(np.int64)).to(DEV) * cache.shape[1]  # noqa: E731
        flat = cache.view(-1)
        for start, size in ((0, data), (bs * data, scale)):
            at = [(page(i) + torch.from_numpy(start + i % bs * size).to(DEV))[:, None] + torch.arange(size, device=DEV) for i in (src, dst)]
            flat[at[1]] = flat[at[0]]
        lens.append(m)
        counts.append(len(dst))
    return moves, np.array(counts, dtype=np.int32), np.array(lens, dtype=np.int32), w_out, p_out, cache


def exact(case, seed):
    st = prepare(case, seed)
    return {"table": _exact_table, "rotary": _exact_rotary, "weights": _exact_weights, "evict": _exact_evict}[case["kind"]](case, st)
