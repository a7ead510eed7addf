"""A cache of bounded size as a server would run it: table, rotation, insert, attention, weights,
eviction, step after step, against plain forms of each step on a host copy of the rows."""
import numpy as np
import pytest
import torch

import oracle
from oracle import attention as plain_attention
from oracle import attn_weights as plain_weights
from oracle import evict as plain_evict
from oracle import rotary as plain_rotary
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu
I32, BF16 = torch.int32, torch.bfloat16
D, ROPE, BS, H, R, WIDTH = 128, 64, 16, 8, 3, 12 * 16
KEEP, FIRST, RECENT = 60, 2, 5


class Server:
    """Device state of R requests, and one step of it."""

    def __init__(self, dev, seed):
        g = np.random.default_rng(seed)
        self.dev, self.rng = dev, g
        stride = -(-BS * oracle.fp8_record_bytes(D, ROPE) // 16) * 16
        self.pages = R * (WIDTH // BS)
        self.cache = torch.zeros((self.pages, stride), dtype=torch.uint8, device=dev)
        self.index_cache = torch.zeros((self.pages, BS * 68), dtype=torch.uint8, device=dev)
        self.table = torch.from_numpy(g.permutation(self.pages).astype(np.int32)).to(dev).view(R, -1)
        self.weights = torch.zeros((R, WIDTH), device=dev)
        self.positions = torch.zeros((R, WIDTH), dtype=I32, device=dev)
        self.lens = torch.zeros(R, dtype=I32, device=dev)
        self.zero = torch.zeros((), device=dev)
        self.keep = torch.full((R,), KEEP, dtype=I32, device=dev)
        self.cos_sin = ops.build_rope_cos_sin_cache(2048, ROPE, scaling="yarn", factor=4.0, original_positions=512, device=dev)
        self.sink = torch.from_numpy(g.standard_normal(H).astype(np.float32)).to(dev)

    def step(self, q, k, index_k, pos, qsl, new):
        """q [T, H, D] and k [T, D] before rotation; pos [T] int64; new [R] tokens of each request."""
        q, k = ops.apply_rotary_embedding(pos, q, self.cos_sin, k)
        seq = self.lens + new
        _, req, slots, _ = ops.compute_slot_mappings(qsl, seq, self.table, BS, q.shape[0])
        ops.quantize_and_insert_k_cache(k, self.cache, slots, BS, rope_dim=ROPE)
        ops.write_indexer_mxfp4_cache(index_k, self.index_cache, slots, BS)
        at = (seq - (qsl[1:] - qsl[:-1]))[req.long()].long() + torch.arange(q.shape[0], device=self.dev) - qsl[req.long()]
        self.positions[req.long(), at] = pos.to(I32)
        self.weights[req.long(), at] = self.zero
        out, lse = ops.chunk_mla_attention(q, self.cache, qsl, seq, req, self.table, BS, rope_dim=ROPE, sink=self.sink)
        back, _ = ops.apply_rotary_embedding(pos, out, self.cos_sin, inverse=True)
        before = self.weights.clone()
        ops.accumulate_attention_weights(q, lse, self.cache, qsl, seq, self.table, BS, self.weights, decay=0.9, sink=self.sink,
                                         rope_dim=ROPE)
        ranked, ranked_pos = self.weights.clone(), self.positions.clone()
        moves, counts, lens, _, _ = ops.select_cache_evictions(self.weights, seq, self.keep, row_positions=self.positions,
                                                               num_first=FIRST, num_recent=RECENT)
        ops.move_cache_rows(self.cache, self.table, moves, counts, BS, D, rope_dim=ROPE)
        ops.move_cache_rows(self.index_cache, self.table, moves, counts, BS, 128, record=ops.PSK_REC_MXFP4)
        self.lens.copy_(lens)
        return q, k, out, lse, back, before, ranked, ranked_pos, seq


def _inputs(rng, dev, new, done):
    T = int(sum(new))
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(BF16).to(dev)  # noqa: E731
    pos = np.concatenate([np.arange(d, d + n) for d, n in zip(done, new)]).astype(np.int64)
    qsl = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return (bf(T, H, D) * 2, bf(T, D), bf(T, 128), torch.from_numpy(pos).to(dev), torch.from_numpy(qsl).to(dev),
            torch.tensor(new, dtype=I32, device=dev))


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _record(rows_bf16, kind):
    """Each row's record by the oracle, in a cache of one row a page."""
    n = len(rows_bf16)
    if kind == "kv":
        c = np.zeros((n, -(-oracle.fp8_record_bytes(D, ROPE) // 16) * 16), np.uint8)
        oracle.quantize_and_insert_k_cache(rows_bf16, np.arange(n), c, 1, D, ROPE)
        return c[:, :D + ROPE], c[:, D + ROPE:D + ROPE + D // 64]
    c = np.zeros((n, 80), np.uint8)
    oracle.write_indexer_mxfp4_cache(rows_bf16, np.arange(n), c, 1, 128)
    return c[:, :64], c[:, 64:68]


def test_decode_over_a_bounded_cache(cuda_device):
    s = Server(cuda_device, 1)
    records = [{} for _ in range(R)]  # position -> (main record, indexer record) of each request
    done = [0] * R
    scale = np.float64(np.float32(D ** -0.5))
    for new in ([90, 61, 7], [1, 1, 1], [5, 0, 1], [1, 30, 1], [1, 1, 60], [2, 1, 1]):
        args = _inputs(s.rng, s.dev, new, done)
        q_in, k_in, index_k = args[:3]
        lens0 = s.lens.cpu().numpy().copy()
        q, k, out, lse, back, before, ranked, ranked_pos, seq = s.step(*args)
        pos, qsl = args[3].cpu().numpy(), args[4].cpu().numpy()
        cs = s.cos_sin.double().cpu().numpy()
        want, tol = plain_rotary.rotate(q_in.double().cpu().numpy(), cs, pos, D - ROPE)
        assert (np.abs(q.double().cpu().numpy() - want) <= tol).all()
        want, tol = plain_rotary.rotate(out.double().cpu().numpy(), cs, pos, D - ROPE, inverse=True)
        assert (np.abs(back.double().cpu().numpy() - want) <= tol).all()
        kv, ix = _record(_bits(k), "kv"), _record(_bits(index_k), "index")
        for r in range(R):
            for t in range(qsl[r], qsl[r + 1]):
                records[r][int(pos[t])] = tuple(x[t] for x in (*kv, *ix))
            done[r] += new[r]
        n = seq.cpu().numpy()
        assert (n == lens0 + np.array(new)).all()
        # the rows before this eviction, from the host's records by their positions
        p = ranked_pos.cpu().numpy()
        host = np.zeros((s.pages, s.cache.shape[1]), np.uint8)
        table = s.table.cpu().numpy()
        for r in range(R):
            for j in range(n[r]):
                page, off = table[r, j // BS], j % BS
                a, b, _, _ = records[r][int(p[r, j])]
                host[page, off * (D + ROPE):(off + 1) * (D + ROPE)] = a
                o = BS * (D + ROPE) + off * (D // 64)
                host[page, o:o + D // 64] = b
        t2r = np.repeat(np.arange(R), new)
        sink = s.sink.cpu().numpy()
        q64 = q.double().cpu().numpy()
        w_out, w_lse, tol, tol_lse = plain_attention.chunk_mla_attention(q64, host, qsl, n, t2r, table, BS, ROPE, scale, sink)
        assert (np.abs(out.double().cpu().numpy() - w_out) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - w_lse) <= tol_lse).all()
        want, tol = plain_weights.accumulate(q64, lse.cpu().numpy(), host, qsl, n, table, BS, ROPE, scale, before.cpu().numpy(), 0.9, sink)
        got = ranked.double().cpu().numpy()
        assert (np.abs(got - want) <= tol + np.abs(want) * 2.0 ** -23).all()  # 0.9 is rounded to binary32
        # the eviction, from the weights it was given
        kept = plain_evict.select(ranked.cpu().numpy(), n, [KEEP] * R, p, FIRST, RECENT)
        lens, now, w = s.lens.cpu().numpy(), s.positions.cpu().numpy(), s.weights.cpu().numpy()
        cache, index_cache = s.cache.cpu().numpy(), s.index_cache.cpu().numpy()
        for r, (moves, m, w2, p2, _) in enumerate(kept):
            assert lens[r] == m == min(n[r], KEEP)
            assert now[r, :m].tolist() == p2 and np.array_equal(w[r, :m], np.array(w2, np.float32))
            assert set(range(FIRST)) <= set(p2) and set(range(done[r] - RECENT, done[r])) <= set(p2)
            for j in range(m):
                page, off = table[r, j // BS], j % BS
                a, b, c, e = records[r][p2[j]]
                assert np.array_equal(cache[page, off * (D + ROPE):(off + 1) * (D + ROPE)], a)
                o = BS * (D + ROPE) + off * (D // 64)
                assert np.array_equal(cache[page, o:o + D // 64], b)
                assert np.array_equal(index_cache[page, off * 64:(off + 1) * 64], c)
                assert np.array_equal(index_cache[page, BS * 64 + off * 4:BS * 64 + (off + 1) * 4], e)


def test_captured_step_is_the_eager_one(cuda_device):
    """One decode step captured and replayed over its own state: the eager steps' bits."""
    eager, graphed = Server(cuda_device, 2), Server(cuda_device, 2)
    prompt = _inputs(np.random.default_rng(5), cuda_device, [70, 80, 66], [0] * R)
    for s in (eager, graphed):
        s.step(*prompt)
        assert s.lens.tolist() == [KEEP] * R
    rng = np.random.default_rng(6)
    steps = [_inputs(rng, cuda_device, [1, 1, 1], [70 + i, 80 + i, 66 + i]) for i in range(4)]
    held = [t.clone() for t in steps[0]]
    state = [graphed.cache, graphed.index_cache, graphed.weights, graphed.positions, graphed.lens]
    saved = [t.clone() for t in state]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(*held)  # warm-up
    torch.cuda.current_stream().wait_stream(side)
    for t, v in zip(state, saved):
        t.copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.step(*held)
    for args in steps:
        want = eager.step(*args)
        for t, v in zip(held, args):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)
        for name in ("cache", "index_cache", "weights", "positions", "lens"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
