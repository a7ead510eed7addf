"""Eviction from a cache on the GPU against plain Python forms (oracle/evict.py): all results
are whole numbers or copies, so everything has to be equal."""
import numpy as np
import pytest
import torch

from oracle import evict as plain
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _i32(a, dev):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def _weights(rng, R, W, kind):
    if kind == "heavy":
        w = np.exp(rng.standard_normal((R, W)) * 3).astype(np.float32)
        w[rng.random((R, W)) < 0.1] = 0
    elif kind == "ties":
        w = rng.integers(0, 4, (R, W)).astype(np.float32)
    elif kind == "same":
        w = np.full((R, W), 0.25, np.float32)
    else:  # every kind of number: both zeros, subnormals, infinities, NaN of both signs
        w = rng.integers(0, 2**32, (R, W), dtype=np.uint32).view(np.float32).copy()
        for v in (0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45):
            w[rng.random((R, W)) < 0.05] = v
        w[rng.random((R, W)) < 0.05] = np.uint32(0xFFC00001).view(np.float32)
    return w


def _select(dev, seed, W, lens, keep, kind="heavy", first=0, recent=0, with_pos=True, place="in"):
    rng = np.random.default_rng(seed)
    R = len(lens)
    w = _weights(rng, R, W, kind)
    p = np.stack([rng.permutation(2 * W)[:W] for _ in range(R)]) if with_pos else None
    want = plain.select(w, lens, keep, p, first, recent)
    gap = 3
    wt = torch.full((R + 1, W + gap), -7.0, device=dev)
    wt[:R, :W] = torch.from_numpy(w)
    pt = torch.full((R + 1, W + gap), -7, dtype=I32, device=dev)
    if with_pos:
        pt[:R, :W] = _i32(p, dev)
    wv, pv = wt[:R, :W], pt[:R, :W] if with_pos else None
    before_w, before_p = wt.clone(), pt.clone()
    kw = {}
    if place == "out":
        kw = dict(weights_out=torch.full((R, W + 1), -3.0, device=dev)[:, 1:], positions_out=torch.full((R, W), -3, dtype=I32, device=dev))
    moves = torch.full((R, W // 2 + 1, 2), -9, dtype=I32, device=dev)
    err = torch.zeros(1, dtype=I32, device=dev)
    mv, nm, out_lens, wo, po = ops.select_cache_evictions(wv, _i32(lens, dev), _i32(keep, dev), row_positions=pv, num_first=first,
                                                          num_recent=recent, moves=moves, err_count=err, **kw)
    assert int(err) == sum(x[4] for x in want)
    assert mv is moves
    got_moves, got_n, got_lens = moves.cpu().numpy(), nm.cpu().numpy(), out_lens.cpu().numpy()
    got_w = wo.cpu().numpy()
    got_p = None if po is None else po.cpu().numpy()
    for r, (ms, m, w2, p2, wide) in enumerate(want):
        assert got_n[r] == len(ms) and got_lens[r] == m, (r, got_n[r], len(ms), got_lens[r], m)
        assert got_moves[r, :len(ms)].tolist() == [list(x) for x in ms]
        assert (got_moves[r, len(ms):] == -9).all()
        if wide:
            continue
        assert np.array_equal(got_w[r, :m].view(np.int32), np.array(w2, np.float32).view(np.int32))
        if got_p is not None:
            assert got_p[r, :m].tolist() == [int(x) for x in p2]
        rest = before_w[r, m:W].cpu().numpy() if place == "in" else np.full(W - m, -3.0, np.float32)
        assert np.array_equal(got_w[r, m:].view(np.int32), rest.view(np.int32))
    if place == "in":  # beside the matrices nothing is written
        assert torch.equal(wt[:, W:], before_w[:, W:]) and torch.equal(wt[R], before_w[R])
        assert torch.equal(pt[:, W:], before_p[:, W:]) and torch.equal(pt[R], before_p[R])
    else:
        assert torch.equal(wt.view(I32), before_w.view(I32)) and torch.equal(pt, before_p)


@pytest.mark.parametrize("W", [1, 2, 31, 32, 33, 100, 1024, 1025, 4096, 4097, 9001, 33000])
@pytest.mark.parametrize("kind", ["heavy", "ties", "any"])
def test_select_sizes(cuda_device, W, kind):
    rng = np.random.default_rng(W)
    lens = [W, max(W - 1, 0), W // 2 + 1 if W > 1 else 1, int(rng.integers(0, W + 1)), 0]
    keep = [W // 2, max(W - 2, 0), W // 3, int(rng.integers(0, W + 1)), 5]
    _select(cuda_device, W, W, lens, keep, kind, first=3, recent=7)
    _select(cuda_device, W + 1, W, lens, keep, kind, place="out", with_pos=W % 2 == 0, first=W % 3, recent=W % 5)


@pytest.mark.parametrize("W,n,keep", [(400001, 400001, 123456), (400001, 399000, 1), (600000, 2, 1), (131072, 131071, 131070)])
def test_select_long(cuda_device, W, n, keep):
    """Beyond the keys that fit in shared memory, and short requests in a wide matrix."""
    _select(cuda_device, 1, W, [n], [keep], "heavy", first=4, recent=64)


def test_select_extremes(cuda_device):
    d = cuda_device
    # all equal; nothing kept; everything kept; lengths below zero; keep below zero; rows without weights
    _select(d, 1, 5000, [5000, 4999, 77, 5000, -3, 5001], [2500, 0, 77, -1, 4, 100], "same", recent=10)
    # more protected rows than are kept: the lower ones
    _select(d, 2, 300, [300, 300], [20, 5], "heavy", first=600, recent=0)
    _select(d, 3, 300, [300, 299], [20, 5], "heavy", first=0, recent=2**31 - 1)
    _select(d, 4, 300, [300], [200], "ties", first=2**31 - 1, recent=2**31 - 1, with_pos=False)
    _select(d, 5, 0, [0, 0], [3, 0])


@pytest.mark.parametrize("seed", range(15))
def test_select_fuzz(cuda_device, seed):
    rng = np.random.default_rng(seed)
    W, R = int(np.exp(rng.uniform(0, np.log(20000)))), int(rng.integers(1, 9))
    lens = rng.integers(0, W + 1, R)
    keep = [int(rng.choice([max(0, n - 1), n // 8, rng.integers(0, W + 1)])) for n in lens]
    _select(cuda_device, 200 + seed, W, lens, keep, str(rng.choice(["heavy", "ties", "any", "same"])),
            int(rng.choice([0, 4])), int(rng.choice([0, 1, 50])), bool(rng.integers(2)), str(rng.choice(["in", "out"])))


def test_select_many_requests(cuda_device):
    _select(cuda_device, 9, 65, [65] * 700, list(range(0, 70)) * 10, "ties", recent=3)


def test_select_lengths_in_place(cuda_device):
    d = cuda_device
    for W in (100, 20000):
        w = torch.rand(3, W, device=d)
        lens, keep = torch.tensor([W, W - 1, 5], dtype=I32, device=d), torch.tensor([W // 2, W // 3, 9], dtype=I32, device=d)
        want = [x.clone() for x in ops.select_cache_evictions(w.clone(), lens, keep)[:3]]
        got = ops.select_cache_evictions(w, lens, keep, seq_lens_out=lens)
        assert got[2].data_ptr() == lens.data_ptr() and torch.equal(lens, want[2]) and torch.equal(got[1], want[1])


RECORDS = [(ops.PSK_REC_FP8_DS_MLA, 512, 64, True, 576, 8), (ops.PSK_REC_FP8_DS_MLA, 64, 0, True, 64, 1),
           (ops.PSK_REC_FP8_DS_MLA, 128, 64, True, 192, 2), (ops.PSK_REC_FP8_DS_MLA, 1024, 128, True, 1152, 16),
           (ops.PSK_REC_FP8_DS_MLA, 512, 64, False, 576, 32), (ops.PSK_REC_FP8_DS_MLA, 1024, 0, False, 1024, 64),
           (ops.PSK_REC_MXFP4, 128, 0, True, 64, 4), (ops.PSK_REC_MXFP4, 32, 0, True, 16, 1), (ops.PSK_REC_MXFP4, 1024, 0, True, 512, 32),
           (ops.PSK_REC_FP8_INDEXER, 128, 0, True, 128, 4)]


@pytest.mark.parametrize("record,D,rope,ue,data,scale", RECORDS)
@pytest.mark.parametrize("bs", [1, 3, 16, 64])
def test_move_records(cuda_device, record, D, rope, ue, data, scale, bs):
    rng = np.random.default_rng(D + bs)
    lens = np.array([150, 37, 1, 0, 90])
    pages = -(-lens // bs)
    table = np.full((5, int(pages.max()) + 2), -1)
    perm, at = rng.permutation(int(pages.sum()) + 3), 0
    for r, n in enumerate(pages):
        table[r, :n] = perm[at:at + n]
        at += n
    base = np.array([0, 2, 0, 1, 5]) if bs > 1 else None
    stride = -(-bs * (data + scale) // 16) * 16 + 32
    cache = rng.integers(0, 256, (len(perm), stride), dtype=np.uint8)
    M, moves, count = 40, np.full((5, 40, 2), -5), np.zeros(5, int)
    shift = np.zeros(5, int) if base is None else base * bs
    for r in range(5):
        m = int(lens[r] * 2 // 3)
        k = min(M, int(lens[r]) - m, m)
        moves[r, :k, 0] = np.sort(rng.permutation(np.arange(m, lens[r]))[:k]) + shift[r]
        moves[r, :k, 1] = np.sort(rng.permutation(m)[:k]) + shift[r]
        count[r] = k
    table[4, 0] = -1  # rows without a page, by a table entry, past the table and past the cache
    if pages[0] > 2:
        table[0, 1] = len(perm) + 9
    moves[1, 0, 0], count[2] = 10**6, -4
    count[0] = M + 7 if count[0] == M else count[0]  # more than there is room for
    want, errors = plain.move(cache, bs, data, scale, table, moves, count, base)
    got, err = torch.from_numpy(cache).to(cuda_device), torch.zeros(1, dtype=I32, device=cuda_device)
    view = got[:, :bs * (data + scale)]
    wide = torch.full((5, M + 2, 2), -1, dtype=I32, device=cuda_device)
    wide[:, :M] = _i32(moves, cuda_device)
    out = ops.move_cache_rows(view, _i32(table, cuda_device), wide[:, :M], _i32(count, cuda_device), bs, D, record=record,
                              rope_dim=rope, is_ue8m0=ue, base_offsets=_i32(base, cuda_device), err_count=err)
    assert out is view and int(err) == errors
    assert np.array_equal(got.cpu().numpy(), want)


def test_move_many(cuda_device):
    """More tiles of moves than CTAs, and a request with far more than the others."""
    rng, bs, R, n = np.random.default_rng(1), 64, 40, 20000
    lens = np.concatenate([[n], rng.integers(1, 700, R - 1)])
    pages = -(-lens // bs)
    table, at = np.full((R, int(pages.max())), -1), 0
    perm = rng.permutation(int(pages.sum()))
    for r, k in enumerate(pages):
        table[r, :k] = perm[at:at + k]
        at += k
    cache = rng.integers(0, 256, (len(perm), bs * 68), dtype=np.uint8)
    w = rng.random((R, n)).astype(np.float32)
    keep = lens // 2
    want_cache = cache
    sel = plain.select(w, lens, keep)
    moves = np.zeros((R, n // 2, 2), int)
    for r, (ms, *_x) in enumerate(sel):
        moves[r, :len(ms)] = np.array(ms).reshape(-1, 2)
    want_cache, _ = plain.move(cache, bs, 64, 4, table, moves, [len(s[0]) for s in sel])
    d = cuda_device
    got = torch.from_numpy(cache).to(d)
    mv, nm, *_ = ops.select_cache_evictions(torch.from_numpy(w).to(d), _i32(lens, d), _i32(keep, d))
    ops.move_cache_rows(got, _i32(table, d), mv, nm, bs, 128, record=ops.PSK_REC_MXFP4)
    assert np.array_equal(got.cpu().numpy(), want_cache)


def test_move_past_4_gib(cuda_device):
    d, bs, stride = cuda_device, 64, 64 * 584
    pages = (1 << 32) // stride + 40
    cache = torch.zeros((pages, stride), dtype=torch.uint8, device=d)
    row = torch.randint(0, 256, (576,), dtype=torch.uint8, device=d)
    cache[pages - 1, 5 * 576:6 * 576] = row
    cache[pages - 1, 64 * 576 + 5 * 8:64 * 576 + 6 * 8] = 77
    table = torch.tensor([[pages - 2, pages - 1]], dtype=I32, device=d)
    moves = torch.tensor([[[69, 3]]], dtype=I32, device=d)
    ops.move_cache_rows(cache, table, moves, torch.ones(1, dtype=I32, device=d), bs, 512)
    assert torch.equal(cache[pages - 2, 3 * 576:4 * 576], row) and int(cache[pages - 2].count_nonzero()) == int(row.count_nonzero()) + 8
    assert int(cache[:pages - 2].any()) == 0


def test_captured_and_on_another_stream(cuda_device):
    d, g = cuda_device, torch.Generator("cuda").manual_seed(1)
    R, W, bs = 6, 9000, 64
    w = torch.rand((R, W), generator=g, device=d)
    table = torch.randperm(R * 141, generator=g, device=d).to(I32).view(R, 141)
    lens, keep = torch.full((R,), W, dtype=I32, device=d), torch.full((R,), 4000, dtype=I32, device=d)
    first = torch.randint(0, 256, (R * 141, bs * 68), dtype=torch.uint8, generator=g, device=d)

    def step(cache, wo):
        mv, nm, ln, _, _ = ops.select_cache_evictions(w, lens, keep, weights_out=wo, num_recent=9)
        ops.move_cache_rows(cache, table, mv, nm, bs, 128, record=ops.PSK_REC_MXFP4)
        return nm, ln

    want_c, want_w = first.clone(), torch.zeros_like(w)
    want = step(want_c, want_w)
    torch.cuda.synchronize(d)
    s = torch.cuda.Stream(d)
    c2, w2 = first.clone(), torch.zeros_like(w)
    s.wait_stream(torch.cuda.current_stream(d))
    with torch.cuda.stream(s):
        step(c2, w2)
    s.synchronize()
    assert torch.equal(c2, want_c) and torch.equal(w2, want_w)
    c3, w3 = first.clone(), torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(c3, w3)
    for _ in range(2):
        c3.copy_(first)
        w3.zero_()
        graph.replay()
        torch.cuda.synchronize(d)
        assert torch.equal(c3, want_c) and torch.equal(w3, want_w)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(cuda_device):
    d = cuda_device
    w, n = torch.zeros(3, 10, device=d), torch.zeros(3, dtype=I32, device=d)
    call = ops.select_cache_evictions
    with pytest.raises(TypeError, match="weights must be"):
        call(w.double(), n, n)
    with pytest.raises(TypeError, match="row_positions"):
        call(w, n, n, row_positions=w)
    with pytest.raises(ValueError, match="at least"):
        call(w[:2], n, n)
    with pytest.raises(ValueError, match="keep_lens"):
        call(w, n, n[:2])
    with pytest.raises(ValueError, match="moves must"):
        call(w, n, n, moves=torch.zeros((3, 4, 2), dtype=I32, device=d))
    with pytest.raises(ValueError, match="side by side"):
        call(w, n, n, moves=torch.zeros((3, 2, 5), dtype=I32, device=d).transpose(1, 2))
    with pytest.raises(ValueError, match="overlap"):
        call(w[:1].expand(3, 10), n, n)
    with pytest.raises(ops.PskError):
        call(w, n, n, num_first=-1)
    with pytest.raises(ops.PskError):
        call(w, n, n, num_moves=n)
    cache = torch.zeros((4, 64 * 584), dtype=torch.uint8, device=d)
    table, mv = torch.zeros((3, 2), dtype=I32, device=d), torch.zeros((3, 5, 2), dtype=I32, device=d)
    with pytest.raises(ops.PskError):
        ops.move_cache_rows(cache, table, mv, n, 64, 500)
    with pytest.raises(ValueError, match="block_table"):
        ops.move_cache_rows(cache, table[:2], mv, n, 64, 512)
    with pytest.raises(TypeError, match="moves must"):
        ops.move_cache_rows(cache, table, mv.float(), n, 64, 512)
