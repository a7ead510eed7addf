"""Attention over paged caches on the GPU against a plain binary64 form, with the
elementwise bounds that form derives (oracle/attention.py)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import attention as plain
from paged_sparse_kv_gb300 import ops, synthetic
from paged_sparse_kv_gb300.pipeline import Pipeline

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_wait_expires(cuda_device):
    """The counter is the device's: other tests may have raised it before."""
    before = ops.device_wait_timeouts()
    yield
    torch.cuda.synchronize()
    assert ops.device_wait_timeouts() == before


def _i32(a, dev):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def _bits(x):
    """binary32 array -> bf16 bit patterns (round to nearest even)."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _cache(rng, pages, bs, D, rope, slack=0, scale=1.0):
    """A cache of N(0, 1) rows times per-row factors around `scale`, every slot filled."""
    stride = -(-bs * oracle.fp8_record_bytes(D, rope) // 16) * 16 + slack
    cache = np.zeros((pages, stride), np.uint8)
    rows = rng.standard_normal((pages * bs, D)) * scale * np.exp2(rng.integers(-2, 3, size=(pages * bs, 1)))
    oracle.quantize_and_insert_k_cache(_bits(rows), np.arange(pages * bs), cache, bs, D, rope)
    return cache


def _query(rng, T, H, D, std, dev, layout="thd"):
    """(device tensor [T, H, D] bf16 of a layout, its binary64 values)."""
    q = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32) * np.float32(std)).to(torch.bfloat16)
    ref = q.double().numpy()
    if layout == "thd":
        return q.to(dev), ref
    if layout == "htd":  # heads outermost
        return q.transpose(0, 1).contiguous().to(dev).transpose(0, 1), ref
    big = torch.full((T, H + 3, D + 24), 7.0, dtype=torch.bfloat16)  # a slice of a wider projection
    big[:, 1:1 + H, 8:8 + D] = q
    return big.to(dev)[:, 1:1 + H, 8:8 + D], ref


def _close(out, lse, want, what=""):
    ref, ref_lse, tol, tol_lse = want
    got = out.double().cpu().numpy()
    gl = lse.double().cpu().numpy()
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    bad = ~nan & ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError(f"{what}: out{tuple(i)} = {got[tuple(i)]}, want {ref[tuple(i)]} +- {tol[tuple(i)]}; "
                             f"{bad.sum()} of {bad.size} beyond their bound")
    fine = np.isfinite(ref_lse)
    assert np.array_equal(np.isnan(gl), np.isnan(ref_lse)), f"{what}: lse"
    assert np.array_equal(gl[np.isinf(ref_lse)], ref_lse[np.isinf(ref_lse)]), f"{what}: lse"
    off = np.abs(gl[fine] - ref_lse[fine])
    assert (off <= tol_lse[fine]).all(), f"{what}: lse off by {off.max()}"


def _indices(rng, T, C, split, cap, xcap, hole):
    """Slots with holes (-1), slots past the caches and repeated ones; one row is empty."""
    idx = rng.integers(0, cap, size=(T, C))
    if split < C:
        idx[:, split:] = rng.integers(0, xcap, size=(T, C - split))
    if C:
        idx[rng.random((T, C)) < hole] = -1
        far = rng.random((T, C)) < hole / 4
        idx[far] = rng.choice([cap, xcap, 2**31 - 1, -2**31, -7], size=int(far.sum()))
        in_a = np.arange(C)[None, :] < split
        lim = np.where(in_a, cap, xcap)
        keep = far & (idx < lim) & (idx >= 0)
        idx[keep] = -1
        if C > 1:
            idx[:, C // 2] = idx[:, 0] if split in (0, C) else idx[:, C // 2]
        if T > 2:
            idx[1] = -1
    return idx.astype(np.int32)


def _run_sparse(dev, seed, T, H, D, rope, C, split, bs=64, xbs=64, sink=True, std=1.0, hole=0.1, layout="thd",
                kscale=1.0, pages=9, xpages=7, scale=None):
    rng = np.random.default_rng(seed)
    a = _cache(rng, pages, bs, D, rope, slack=16, scale=kscale)
    b = _cache(rng, xpages, xbs, D, rope, slack=0, scale=kscale) if split < C else None
    idx = _indices(rng, T, C, split, pages * bs, xpages * xbs, hole)
    q, q64 = _query(rng, T, H, D, std, dev, layout)
    s = rng.standard_normal(H).astype(np.float32) * 2 if sink else None
    scale = D ** -0.5 if scale is None else scale
    want = plain.sparse_mla_attention(q64, a, idx, bs, rope, np.float32(scale).astype(np.float64), s, b, xbs, split)
    wide = torch.full((T, C + 5), -1, dtype=torch.int32, device=dev)
    wide[:, 3:3 + C] = torch.from_numpy(idx).to(dev)
    big = torch.full((T + 2, H + 1, D + 8), -3.0, dtype=torch.bfloat16, device=dev)
    out = big[1:1 + T, :H, 8:]
    blse = torch.full((T + 2, H + 3), -3.0, device=dev)
    got = ops.sparse_mla_attention(q, torch.from_numpy(a).to(dev), wide[:, 3:3 + C], bs,
                                   extra_cache=None if b is None else torch.from_numpy(b).to(dev),
                                   extra_block_size=xbs, split=split, softmax_scale=scale,
                                   sink=None if s is None else torch.from_numpy(s).to(dev), rope_dim=rope,
                                   out=out, lse=blse[1:1 + T, 2:2 + H])
    assert got[0].data_ptr() == out.data_ptr()
    _close(out, blse[1:1 + T, 2:2 + H], want, f"T {T} H {H} D {D} C {C}")
    # nothing around the outputs is written
    out.fill_(-3.0)
    blse[1:1 + T, 2:2 + H] = -3.0
    assert bool((big == -3.0).all()) and bool((blse == -3.0).all())


@pytest.mark.parametrize("T,H,C,split", [
    (1, 1, 1, 1), (1, 16, 640, 128), (3, 7, 5, 5), (2, 64, 127, 127), (2, 64, 128, 128), (2, 64, 129, 128),
    (5, 24, 200, 37), (2, 128, 640, 128), (3, 65, 300, 0), (2, 130, 257, 100), (1, 33, 1152, 128), (7, 8, 64, 0),
    (2, 17, 130, 130), (1, 128, 2300, 200)])
def test_sparse_shapes(cuda_device, T, H, C, split):
    _run_sparse(cuda_device, 1000 * T + H + C, T, H, 512, 64, C, split)


@pytest.mark.parametrize("D,rope", [(512, 0), (512, 128), (512, 448), (256, 64), (256, 0), (256, 192),
                                    (128, 64), (128, 0)])
@pytest.mark.parametrize("H", [5, 64])
def test_sparse_record_shapes(cuda_device, D, rope, H):
    _run_sparse(cuda_device, D + rope + H, 3, H, D, rope, 333, 100)


@pytest.mark.parametrize("seed", range(16))
def test_sparse_fuzz(cuda_device, seed):
    rng = np.random.default_rng(seed)
    D = int(rng.choice([128, 256, 512]))
    C = int(rng.choice([rng.integers(1, 40), rng.integers(100, 700)]))
    _run_sparse(cuda_device, 50 + seed, T=int(rng.integers(1, 9)), H=int(rng.integers(1, 130)), D=D,
                rope=int(rng.choice([0, 64])), C=C, split=int(rng.integers(0, C + 1)), bs=int(rng.choice([1, 3, 16, 64])),
                xbs=int(rng.choice([2, 5, 64])), sink=bool(rng.integers(0, 2)), hole=float(rng.choice([0.0, 0.1, 0.9])),
                layout=str(rng.choice(["thd", "htd", "slice"])), pages=40, xpages=50)


@pytest.mark.parametrize("std,kscale", [(30.0, 1.0), (1.0, 1e-3), (1e-3, 1.0), (4.0, 300.0), (1.0, 1e4)])
def test_sparse_magnitudes(cuda_device, std, kscale):
    """Nearly one-hot and nearly even weights, scores into the thousands, a
    running maximum that grows in steps of any size."""
    _run_sparse(cuda_device, 77, 4, 40, 512, 64, 700, 300, std=std, kscale=kscale)


def test_sparse_many_tokens(cuda_device):
    """More units of work than CTAs can run at once, odd numbers of everything."""
    _run_sparse(cuda_device, 5, 401, 9, 128, 64, 150, 31)
    _run_sparse(cuda_device, 6, 200, 66, 512, 64, 129, 65)


@pytest.mark.parametrize("T,H,D,C", [(160, 9, 128, 700), (60, 130, 512, 600), (153, 64, 256, 2000)])
def test_sparse_last_units_cut(cuda_device, T, H, D, C):
    """A few more units than CTAs: the last ones are cut along their columns and joined."""
    _run_sparse(cuda_device, T + H, T, H, D, 64, C, C // 3)


@pytest.mark.parametrize("T,H,D,C,sink", [
    (64, 64, 512, 640, True), (76, 33, 256, 300, False), (1, 16, 512, 1000, True), (3, 5, 128, 1024, False),
    (8, 16, 512, 640, True), (30, 128, 512, 300, True), (52, 130, 128, 257, True), (2, 1, 256, 129, True)])
def test_sparse_joined_in_cluster(cuda_device, T, H, D, C, sink):
    """Two parts of a unit, or up to eight of 16 columns, joined through shared memory."""
    _run_sparse(cuda_device, T + H + C, T, H, D, 64, C, C // 5, sink=sink, hole=0.5)


def test_sparse_joined_in_cluster_captured(cuda_device):
    """Captured, replayed, and run beside another call of its kind: the eager call's bits."""
    d = cuda_device
    cases = [_decode_case(d, 30, T=64), _decode_case(d, 31, T=1, H=16)]
    want = [ops.sparse_mla_attention(q, c, i, 64) for q, c, i in cases]
    torch.cuda.synchronize(d)
    graphs, outs = [], []
    for q, c, i in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.sparse_mla_attention(q, c, i, 64))
        graphs.append(g)
    streams = [torch.cuda.Stream(d), torch.cuda.Stream(d)]
    for _ in range(3):
        for s, g, o in zip(streams, graphs, outs):
            o[0].fill_(-3.0)
            s.wait_stream(torch.cuda.current_stream(d))
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize(d)
        for (a, b), (x, y) in zip(want, outs):
            assert torch.equal(a, x) and torch.equal(b, y)


def test_sparse_growing_scores(cuda_device):
    """Scores that grow from the first column to the last, so that every tile
    raises the maximum, by little and by more than any lazy threshold."""
    d = cuda_device
    D, H, n = 512, 64, 1024
    for step in (0.02, 0.5):
        rows = np.zeros((n, D))
        rows[:, 0] = np.arange(n) * step
        rows[:, 1:] = np.random.default_rng(1).standard_normal((n, D - 1))
        cache = np.zeros((n // 64, 64 * 584), np.uint8)
        oracle.quantize_and_insert_k_cache(_bits(rows), np.arange(n), cache, 64, D, 64)
        q64 = np.zeros((2, H, D))
        q64[:, :, 0] = np.linspace(-1, 1, H) * 1.0
        q = torch.from_numpy(q64).to(torch.bfloat16)
        idx = np.stack([np.arange(n), np.arange(n)[::-1]]).astype(np.int32)
        want = plain.sparse_mla_attention(q.double().numpy(), cache, idx, 64, 64, 1.0)
        got = ops.sparse_mla_attention(q.to(d), torch.from_numpy(cache).to(d), _i32(idx, d), 64, softmax_scale=1.0)
        _close(*got, want, f"step {step}")


def test_sparse_nothing_visible(cuda_device):
    """No columns, all columns -1, an empty sink and an infinite one."""
    d = cuda_device
    rng = np.random.default_rng(2)
    cache = torch.from_numpy(_cache(rng, 2, 64, 512, 64)).to(d)
    q, _ = _query(rng, 3, 20, 512, 1.0, d)
    for C in (0, 1, 130):
        idx = torch.full((3, C), -1, dtype=torch.int32, device=d)
        for sink in (None, torch.zeros(20, device=d)):
            out, lse = ops.sparse_mla_attention(q, cache, idx, 64, sink=sink)
            assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    idx = torch.arange(9, dtype=torch.int32, device=d)[None, :].expand(3, 9).contiguous()
    base, lse0 = ops.sparse_mla_attention(q, cache, idx, 64)
    out, lse = ops.sparse_mla_attention(q, cache, idx, 64, sink=torch.full((20,), -float("inf"), device=d))
    assert torch.equal(out, base) and torch.equal(lse, lse0)
    out, lse = ops.sparse_mla_attention(q, cache, idx, 64, sink=torch.full((20,), float("inf"), device=d))
    assert bool((out == 0).all()) and torch.equal(lse, lse0)


def test_sparse_nan_rows(cuda_device):
    """Rows of NaN and infinity: without effect where no column names them, what
    the formulas give where one does."""
    d = cuda_device
    rng = np.random.default_rng(3)
    cache = _cache(rng, 4, 64, 512, 64)
    cache[1, :64 * 576] = 0x7F          # page 1: NaN codes and NaN rope values
    cache[2, 64 * 576:] = 0xFF          # page 2: scale 2^128
    q, q64 = _query(rng, 4, 30, 512, 1.0, d)
    idx = np.concatenate([np.arange(64), 192 + np.arange(64)] * 2)[None, :].repeat(4, 0).astype(np.int32)
    idx[1, 200] = 70                    # a row of NaN
    idx[2, 5] = 128 + 3                 # a row of infinities and NaN (0 * 2^128)
    got = ops.sparse_mla_attention(q, torch.from_numpy(cache).to(d), _i32(idx, d), 64)
    want = plain.sparse_mla_attention(q64, cache, idx, 64, 64, 512 ** -0.5)
    assert np.isnan(want[0][1]).all() and not np.isnan(want[0][[0, 3]]).any()
    o = got[0].double().cpu().numpy()
    assert np.isnan(o[1]).all() and np.isnan(o[2]).all()
    _close(got[0][[0, 3]], got[1][[0, 3]], [w[[0, 3]] for w in want])
    # a NaN query touches its own head alone
    q[3, 7, 100] = float("nan")
    again = ops.sparse_mla_attention(q, torch.from_numpy(cache).to(d), _i32(idx, d), 64)[0]
    assert bool(torch.isnan(again[3, 7]).all())
    keep = torch.ones(30, dtype=torch.bool, device=d)
    keep[7] = False
    assert torch.equal(again[3, keep], got[0][3, keep]) and torch.equal(again[0], got[0][0])


def test_sparse_subnormal_and_large_scales(cuda_device):
    """Every UE8M0 scale that gives finite rows: products that round, underflow
    or are subnormal in bf16 are those of the gather."""
    d = cuda_device
    rng = np.random.default_rng(4)
    cache = _cache(rng, 4, 64, 128, 0)
    sc = cache[:, 64 * 128:64 * 130].reshape(4 * 64, 2)
    sc[:, 0] = np.arange(256) % 120     # down to 2^-127
    sc[:, 1] = 0
    cache[:, 64 * 128:64 * 130] = sc.reshape(4, -1)
    q, q64 = _query(rng, 2, 16, 128, 1.0, d)
    idx = np.stack([np.arange(120), np.arange(119, -1, -1)]).astype(np.int32)
    got = ops.sparse_mla_attention(q, torch.from_numpy(cache).to(d), _i32(idx, d), 64, rope_dim=0)
    _close(*got, plain.sparse_mla_attention(q64, cache, idx, 64, 0, np.float64(np.float32(128 ** -0.5))))
    one = ops.sparse_mla_attention(q, torch.from_numpy(cache).to(d), _i32(np.full((2, 1), 7), d), 64, rope_dim=0)[0]
    row = torch.from_numpy(plain.rows_of(cache, 64, 128, 0, [7])).to(d)
    assert torch.equal(one.double(), row[None].expand(2, 16, 128))


def test_sparse_far_pages(cuda_device):
    """Records past byte 2^32 of a cache, odd page size."""
    d = cuda_device
    D, rope, bs = 512, 64, 3
    stride = 1760
    pages = (1 << 32) // stride + 900
    cache = torch.zeros((pages, stride), dtype=torch.uint8, device=d)
    rng = np.random.default_rng(6)
    few = _cache(rng, 60, bs, D, rope)
    where = np.sort(rng.choice(np.arange(pages - 800, pages), size=60, replace=False))
    cache[torch.from_numpy(where).to(d), :few.shape[1]] = torch.from_numpy(few).to(d)
    local = rng.integers(0, 180, size=(3, 170)).astype(np.int32)
    idx = (where[local // bs] * bs + local % bs).astype(np.int32)
    q, q64 = _query(rng, 3, 20, D, 1.0, d)
    got = ops.sparse_mla_attention(q, cache, _i32(idx, d), bs)
    _close(*got, plain.sparse_mla_attention(q64, few, local, bs, rope, np.float64(np.float32(D ** -0.5))))
    table = np.full((1, 60), -1, np.int32)
    table[0] = where
    got = ops.chunk_mla_attention(q[:2], cache, _i32([0, 2], d), _i32([180], d), _i32([0, 0], d), _i32(table, d), bs)
    near = np.arange(60, dtype=np.int32)[None, :]
    _close(*got, plain.chunk_mla_attention(q64[:2], few, [0, 2], [180], [0, 0], near, bs, rope,
                                           np.float64(np.float32(D ** -0.5))))


def _run_chunk(dev, seed, q_lens, prefix, H, D, rope, bs, window, sink=True, with_replay=False, with_base=False,
               with_valid=False, missing=0.0, pad=0, std=1.0, layout="thd"):
    rng = np.random.default_rng(seed)
    q_lens, prefix = np.array(q_lens), np.array(prefix)
    R, T = len(q_lens), int(q_lens.sum()) + pad
    seq = (q_lens + prefix).astype(np.int32)
    qsl = np.concatenate([[0], np.cumsum(q_lens)])
    t2r = np.concatenate([np.repeat(np.arange(R), q_lens), np.full(pad, R)]).astype(np.int32)
    width = max(1, -(-int(seq.max()) // bs))
    pages = max(R * width, 4)
    table = rng.permutation(pages)[:R * width].reshape(R, width).astype(np.int32)
    table[rng.random((R, width)) < missing] = -1
    base = rng.integers(0, 2, size=R).astype(np.int32) if with_base else None
    replay = rng.integers(0, int(seq.max()) + 1, size=R).astype(np.int32) if with_replay else None
    valid = rng.random(T) < 0.8 if with_valid else None
    cache = _cache(rng, pages, bs, D, rope)
    q, q64 = _query(rng, T, H, D, std, dev, layout)
    s = rng.standard_normal(H).astype(np.float32) if sink else None
    scale = np.float64(np.float32(D ** -0.5))
    want = plain.chunk_mla_attention(q64, cache, qsl, seq, t2r, table, bs, rope, scale, s, window, replay, base, valid)
    got = ops.chunk_mla_attention(
        q, torch.from_numpy(cache).to(dev), _i32(qsl, dev), _i32(seq, dev), _i32(t2r, dev), _i32(table, dev), bs,
        window_size=window, replay_start=_i32(replay, dev), base_offsets=_i32(base, dev),
        is_valid_token=None if valid is None else torch.from_numpy(valid).to(dev),
        sink=None if s is None else torch.from_numpy(s).to(dev), rope_dim=rope)
    _close(*got, want, f"q {q_lens} prefix {prefix} H {H} D {D} window {window}")


@pytest.mark.parametrize("q_lens,prefix,H,window", [
    ([1], [0], 1, 0), ([1], [127], 16, 0), ([1], [128], 16, 0), ([1, 1, 1], [5, 300, 0], 64, 0), ([9], [0], 16, 0),
    ([130], [3], 8, 0), ([5, 0, 33], [200, 9, 1], 16, 128), ([4], [1000], 64, 128), ([3], [700], 128, 0),
    ([1, 1], [3000, 2000], 20, 0), ([40], [60], 4, 1), ([17, 2], [0, 90], 1, 33), ([21], [40], 70, 7)])
def test_chunk_shapes(cuda_device, q_lens, prefix, H, window):
    _run_chunk(cuda_device, sum(q_lens) + H, q_lens, prefix, H, 512, 64, 64, window)


@pytest.mark.parametrize("seed", range(20))
def test_chunk_fuzz(cuda_device, seed):
    rng = np.random.default_rng(900 + seed)
    R = int(rng.integers(1, 6))
    _run_chunk(cuda_device, seed, rng.integers(0, 30, size=R) + (np.arange(R) == 0), rng.integers(0, 400, size=R),
               H=int(rng.choice([1, 2, 5, 8, 16, 20, 32, 48, 64, 100])), D=int(rng.choice([128, 256, 512])),
               rope=int(rng.choice([0, 64])), bs=int(rng.choice([1, 7, 16, 64])),
               window=int(rng.choice([0, 1, 50, 128, 300])), sink=bool(rng.integers(0, 2)),
               with_replay=bool(rng.integers(0, 2)), with_base=bool(rng.integers(0, 2)),
               with_valid=bool(rng.integers(0, 2)), missing=float(rng.choice([0.0, 0.2, 1.0])),
               pad=int(rng.choice([0, 3])), std=float(rng.choice([0.5, 6.0])),
               layout=str(rng.choice(["thd", "htd", "slice"])))


def test_chunk_decode_batch_of_many_requests(cuda_device):
    """Neighbouring tokens of different requests, more of them than fit at once."""
    rng = np.random.default_rng(8)
    _run_chunk(cuda_device, 8, [1] * 300, rng.integers(0, 200, size=300), 16, 128, 64, 16, 128)
    _run_chunk(cuda_device, 9, [1] * 40, rng.integers(0, 500, size=40), 8, 512, 64, 64, 0)


@pytest.mark.parametrize("q_lens,prefix,H,D,window", [
    ([64, 9, 0, 40], [3000, 1500, 5, 10], 16, 128, 0), ([50, 21], [2500, 40], 5, 256, 2000),
    ([40, 40], [1100, 1800], 32, 128, 0), ([1] * 40, list(range(0, 3000, 75)), 70, 128, 0),
    ([8] * 30, list(range(0, 2400, 80)), 8, 128, 1100)])
def test_chunk_units_cut(cuda_device, q_lens, prefix, H, D, window):
    """Units of one and of several tokens, cut along their positions and joined."""
    _run_chunk(cuda_device, H + D, q_lens, prefix, H, D, 64, 64, window, pad=3, missing=0.05)


@pytest.mark.parametrize("what", ["scale 247", "scale 255", "byte", "rope nan", "rope inf"])
@pytest.mark.parametrize("H", [1, 8, 33])
def test_chunk_non_finite_rows(cuda_device, what, H):
    """Every way a record can hold a NaN or an infinity: only tokens that see it notice."""
    d = cuda_device
    rng = np.random.default_rng(13)
    D, bs, bad = 256, 16, 53
    cache = _cache(rng, 8, bs, D, 64)
    rec, at = D + 64, bad % bs
    page = cache[bad // bs]
    scales = page[bs * rec + at * (D // 64):]
    if what.startswith("scale"):
        page[at * rec + 3] = 0xFE          # -448
        scales[0] = int(what.split()[1])
    elif what == "byte":
        page[at * rec + 130] = 0xFF
    else:
        page[at * rec + D - 64 + 6:at * rec + D - 64 + 8] = (0xC1, 0x7F) if what == "rope nan" else (0x80, 0xFF)
    q, q64 = _query(rng, 40, H, D, 1.0, d)
    args = ([0, 40], [75], np.zeros(40, np.int32), np.arange(8, dtype=np.int32)[None, :])  # positions 35 ... 74
    with np.errstate(all="ignore"):
        want = plain.chunk_mla_attention(q64, cache, *args, bs, 64, np.float64(np.float32(D ** -0.5)), window=10)
    out, lse = ops.chunk_mla_attention(q, torch.from_numpy(cache).to(d), *(_i32(a, d) for a in args), bs, window_size=10)
    sees = (np.arange(35, 75) >= bad) & (np.arange(35, 75) < bad + 10)
    dark = torch.from_numpy(~sees).to(d)
    _close(out[dark], lse[dark], [w[~sees] for w in want], f"H {H} {what}")
    assert bool((~torch.isfinite(out[~dark].float())).any((1, 2)).all())


def test_chunk_more_new_tokens_than_positions(cuda_device):
    """seq_lens below the query length: the first tokens lie before position 0."""
    d = cuda_device
    rng = np.random.default_rng(10)
    cache = _cache(rng, 4, 16, 128, 0)
    q, q64 = _query(rng, 9, 6, 128, 1.0, d)
    args = ([0, 9], [5], np.zeros(9, np.int32), np.arange(4, dtype=np.int32)[None, :])
    want = plain.chunk_mla_attention(q64, cache, *args, 16, 0, np.float64(np.float32(128 ** -0.5)))
    got = ops.chunk_mla_attention(q, torch.from_numpy(cache).to(d), *(_i32(a, d) for a in args), 16, rope_dim=0)
    _close(*got, want)
    assert bool((got[0][:4] == 0).all()) and bool((got[0][4] != 0).any())


def test_chunk_nan_row_touches_those_that_see_it(cuda_device):
    """Tokens side by side, some of which see a NaN row and some do not."""
    d = cuda_device
    rng = np.random.default_rng(11)
    for H in (1, 8, 64):
        cache = _cache(rng, 8, 16, 512, 64)
        cache[3, 5 * 576:6 * 576] = 0x7F    # position 53 of the request
        q, q64 = _query(rng, 40, H, 512, 1.0, d)
        args = ([0, 40], [75], np.zeros(40, np.int32), np.arange(8, dtype=np.int32)[None, :])  # positions 35 ... 74
        want = plain.chunk_mla_attention(q64, cache, *args, 16, 64, np.float64(np.float32(512 ** -0.5)), window=10)
        got = ops.chunk_mla_attention(q, torch.from_numpy(cache).to(d), *(_i32(a, d) for a in args), 16, window_size=10)
        seen = np.isnan(want[0]).all((1, 2))
        assert seen.sum() == 10
        _close(*got, want, f"H {H}")


def test_forms_agree(cuda_device):
    """The position form equals the index form over the slots of its positions."""
    d = cuda_device
    rng = np.random.default_rng(12)
    cache = torch.from_numpy(_cache(rng, 30, 16, 512, 64)).to(d)
    q, _ = _query(rng, 50, 64, 512, 1.0, d)
    qsl, seq = _i32([0, 20, 50], d), _i32([100, 200], d)
    t2r = _i32([0] * 20 + [1] * 30, d)
    table = _i32(rng.permutation(30)[:26].reshape(2, 13), d)
    idx, _ = ops.decode_swa_indices_and_lens(qsl, seq, t2r, table, 16, 128)
    a = ops.sparse_mla_attention(q, cache, idx, 16)
    b = ops.chunk_mla_attention(q, cache, qsl, seq, t2r, table, 16, window_size=128)
    # the same visible rows in the same order: equal up to where the tiles begin
    assert torch.allclose(a[0].float(), b[0].float(), rtol=2**-6, atol=2**-8)
    assert torch.allclose(a[1], b[1], rtol=1e-5, atol=1e-5)


def test_refusals(cuda_device):
    d = cuda_device
    cache = torch.zeros((4, 64 * 584), dtype=torch.uint8, device=d)
    q = torch.zeros((2, 8, 512), dtype=torch.bfloat16, device=d)
    idx = torch.zeros((2, 16), dtype=torch.int32, device=d)
    bad = [dict(q=q.float()), dict(indices=idx.long()), dict(indices=idx[:1]), dict(q=q[0]),
           dict(q=q.cpu()), dict(out=torch.zeros_like(q)[:, :4]), dict(sink=torch.zeros(4, device=d)),
           dict(sink=torch.zeros(8, device=d, dtype=torch.float64)), dict(lse=torch.zeros((2, 7), device=d)),
           dict(workspace=torch.zeros(16, device=d)), dict(q=q.transpose(1, 2))]
    for kw in bad:
        a = dict(q=q, cache=cache, indices=idx, block_size=64)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            ops.sparse_mla_attention(**a)
    for kw in (dict(rope_dim=32), dict(split=17), dict(split=3), dict(softmax_scale=0.0), dict(block_size=65),
               dict(q=q[:, :, :64].contiguous(), rope_dim=0), dict(out=q.as_strided((2, 8, 512), (8, 8, 1)))):
        a = dict(q=q, cache=cache, indices=idx, block_size=64)
        a.update(kw)
        with pytest.raises(ops.PskError):
            ops.sparse_mla_attention(**a)
    z, qsl = torch.zeros(2, dtype=torch.int32, device=d), torch.tensor([0, 2], dtype=torch.int32, device=d)
    table = torch.zeros((1, 4), dtype=torch.int32, device=d)
    args = (q, cache, qsl, z[:1], z, table, 64)
    ops.chunk_mla_attention(*args)
    for i, x in ((2, qsl.long()), (2, qsl[:1]), (3, z.float()), (4, z[:1]), (5, table[:0]), (5, table.long())):
        bad = list(args)
        bad[i] = x
        with pytest.raises((TypeError, ValueError)):
            ops.chunk_mla_attention(*bad)
    with pytest.raises(ops.PskError):
        ops.chunk_mla_attention(*args, window_size=-1)
    empty = ops.sparse_mla_attention(q[:0], cache, idx[:0], 64)
    assert empty[0].shape == (0, 8, 512) and empty[1].shape == (0, 8)


def _decode_case(d, seed, T=24, H=64, C=640):
    rng = np.random.default_rng(seed)
    cache = torch.from_numpy(_cache(rng, 40, 64, 512, 64)).to(d)
    q, _ = _query(rng, T, H, 512, 1.0, d)
    idx = _i32(rng.integers(-5, 40 * 64, size=(T, C)), d)
    return q, cache, idx


def test_repeatable_and_on_streams(cuda_device):
    """The same bits from every call: eager, on side streams at the same time
    (each with its own scratch), and from two captured graphs in any order."""
    d = cuda_device
    cases = [_decode_case(d, 20), _decode_case(d, 21, T=3, H=16, C=2000)]
    want = [ops.sparse_mla_attention(q, c, i, 64) for q, c, i in cases]
    torch.cuda.synchronize(d)
    streams = [torch.cuda.Stream(d) for _ in cases]
    for _ in range(20):
        got = []
        for s, (q, c, i) in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(ops.sparse_mla_attention(q, c, i, 64))
        torch.cuda.synchronize(d)
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for q, c, i in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.sparse_mla_attention(q, c, i, 64))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize(d)
        for k in set(order):
            assert torch.equal(outs[k][0], want[k][0]) and torch.equal(outs[k][1], want[k][1])
    # one scratch buffer for calls that follow each other on a stream
    need = max(ops.sparse_mla_attention_workspace_bytes(d, q.shape[0], q.shape[1], 512, i.shape[1])
               for q, _, i in cases)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=d)
    for q, c, i in cases * 2:
        k = 0 if q.shape[0] == 24 else 1
        g = ops.sparse_mla_attention(q, c, i, 64, workspace=ws)
        assert torch.equal(g[0], want[k][0]) and torch.equal(g[1], want[k][1])


def test_inputs_written_just_before(cuda_device):
    """Every input written by an ordinary kernel right before the call is seen."""
    d = cuda_device
    a, b = _decode_case(d, 30), _decode_case(d, 31)
    live = [x.clone() for x in a]
    want = [ops.sparse_mla_attention(q, c, i, 64)[0] for q, c, i in (a, b)]
    torch.cuda.synchronize(d)
    for k in range(30):
        for dst, src in zip(live, (a, b)[k % 2]):
            torch.add(src, 0, out=dst)
        got = ops.sparse_mla_attention(live[0], live[1], live[2], 64)[0]
        assert torch.equal(got, want[k % 2])


@pytest.mark.parametrize("name", ["tiny", "decode"])
def test_step_from_lengths_to_attention(cuda_device, name):
    """A serving step from request lengths alone: block tables, slot maps, the
    insert, the index build, and attention over both caches."""
    d = cuda_device
    w = synthetic.make(name)
    p = Pipeline(w, d)
    p.fill_caches_with_quantized_rows(seed=9)
    bs, T, D, rope, W = w.swa_cache.block_size, w.num_tokens, w.head_dim, w.rope_dim, w.window
    H = 24
    rng = np.random.default_rng(13)
    pool = _i32(rng.permutation(w.swa_cache.num_pages), d)
    table = torch.empty_like(p.swa_bt)
    # a table for the contexts before this step, then grown by the new tokens
    old = p.seq_lens - (p.qsl[1:] - p.qsl[:-1])
    _, counts, head = ops.extend_block_tables(old.contiguous(), pool, table, bs)
    err = torch.zeros(1, dtype=torch.int32, device=d)
    _, counts, head = ops.extend_block_tables(p.seq_lens, pool, table, bs, page_counts=counts, pool_head=head,
                                              err_count=err)
    pos, t2r, slots, _ = ops.compute_slot_mappings(p.qsl, p.seq_lens, table, bs, T)
    assert int(err) == 0 and int(head) == int(((p.seq_lens + bs - 1) // bs).sum())
    assert torch.equal(t2r, p.t2r)
    ops.quantize_and_insert_k_cache(p.k, p.swa_cache, slots, bs, rope_dim=rope)
    comp_bt = p.comp_bt if p.comp_bt is not None else table
    idx, lens = ops.combine_topk_swa_indices(p.qsl, p.seq_lens, t2r, p.replay, table, bs, comp_bt,
                                             w.comp_cache.block_size, W, w.compress_ratio, p.topk)
    q, q64 = _query(rng, T, H, D, 1.0, d)
    sink = torch.randn(H, device=d)
    got = ops.sparse_mla_attention(q, p.swa_cache, idx, bs, extra_cache=p.comp_cache,
                                   extra_block_size=w.comp_cache.block_size, split=W, sink=sink, rope_dim=rope)
    scale = np.float64(np.float32(D ** -0.5))
    want = plain.sparse_mla_attention(q64, p.swa_cache.cpu().numpy(), idx.cpu().numpy(), bs, rope, scale,
                                      sink.cpu().numpy(), p.comp_cache.cpu().numpy(), w.comp_cache.block_size, W)
    _close(*got, want, name)
    # the window part alone, straight from the positions
    got = ops.chunk_mla_attention(q, p.swa_cache, p.qsl, p.seq_lens, t2r, table, bs, window_size=W,
                                  replay_start=p.replay, rope_dim=rope)
    want = plain.sparse_mla_attention(q64, p.swa_cache.cpu().numpy(), idx[:, :W].cpu().numpy(), bs, rope, scale)
    _close(*got, want, name + " window")
