"""Attention weights per cached row on the GPU against a plain binary64 form, with the bounds it
derives (oracle/attn_weights.py)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import attn_weights as plain
from oracle.attention import rows_of
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu
I32, BF16 = torch.int32, torch.bfloat16


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
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(BF16).view(torch.int16).numpy().view(np.uint16)


def _cache(rng, pages, bs, D, rope, slack=0):
    stride = -(-bs * oracle.fp8_record_bytes(D, rope) // 16) * 16 + slack
    cache = np.zeros((pages, stride), np.uint8)
    rows = rng.standard_normal((pages * bs, D)) * np.exp2(rng.integers(-2, 3, size=(pages * bs, 1)))
    oracle.quantize_and_insert_k_cache(_bits(rows), np.arange(pages * bs), cache, bs, D, rope)
    return cache


def _query(rng, T, H, D, std, dev, layout):
    q = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32) * np.float32(std)).to(BF16)
    ref = q.double().numpy()
    if layout == "htd":
        return q.transpose(0, 1).contiguous().to(dev).transpose(0, 1), ref
    if layout == "slice":
        big = torch.full((T, H + 3, D + 24), 7.0, dtype=BF16)
        big[:, 1:1 + H, 8:8 + D] = q
        return big.to(dev)[:, 1:1 + H, 8:8 + D], ref
    return q.to(dev), ref


def _close(got, want, tol, what=""):
    g = got.double().cpu().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN in other places"
    bad = ~nan & ~(np.abs(g - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}{i}: {g[i]}, want {want[i]} +- {tol[i]}; {bad.sum()} of {bad.size}")


def _lse(q64, cache, bs, rope, table, seq, qsl, base, scale, rng):
    """About what the attention returns: the log of the sum over all rows of the request."""
    T, H, D = q64.shape
    lse = np.zeros((T, H), np.float32)
    for r in range(len(seq)):
        slots = [int(table[r, i]) * bs + o for i in range(table.shape[1]) if table[r, i] >= 0 for o in range(bs)][:max(int(seq[r]), 1)]
        k = rows_of(cache, bs, D, rope, slots)
        for t in range(int(qsl[r]), min(int(qsl[r + 1]), T)):
            if len(slots):
                s = q64[t] @ k.T * scale
                lse[t] = s.max(1) + np.log(np.exp(s - s.max(1)[:, None]).sum(1))
    return lse + rng.standard_normal((T, H)).astype(np.float32) * 0.1


def _run(dev, seed, q_lens, prefix, H, D=512, rope=64, bs=64, window=0, sink=True, replay=False, base=False, valid=False,
         missing=0.0, pad=0, std=1.0, layout="thd", decay=1.0, place="out", narrow=0):
    rng = np.random.default_rng(seed)
    q_lens, prefix = np.array(q_lens), np.array(prefix)
    R, T = len(q_lens), int(q_lens.sum()) + pad
    seq = q_lens + prefix
    qsl = np.concatenate([[0], np.cumsum(q_lens)])
    width = max(1, -(-int(seq.max()) // bs))
    pages = max(R * width, 4)
    table = rng.permutation(pages)[:R * width].reshape(R, width).astype(np.int32)
    table[rng.random((R, width)) < missing] = -1
    off = rng.integers(0, 2, size=R) if base else None
    rep = rng.integers(0, int(seq.max()) + 1, size=R) if replay else None
    ok = rng.random(T) < 0.8 if valid else None
    cache = _cache(rng, pages, bs, D, rope, slack=16)
    q, q64 = _query(rng, T, H, D, std, dev, layout)
    s = rng.standard_normal(H).astype(np.float32) if sink else None
    scale = np.float64(np.float32(D ** -0.5))
    lse = _lse(q64, cache, bs, rope, table, seq, qsl, off, scale, rng)
    if T > 2:
        lse[1, 0] = -np.inf  # a (token, head) that saw nothing
    W = max(1, int(seq.max()) - narrow)
    w = rng.random((R, W)).astype(np.float32) * 3
    want, tol = plain.accumulate(q64, lse, cache, qsl, seq, table, bs, rope, scale, w, decay, s, window, rep, off, ok)
    big = torch.full((R + 1, W + 5), -3.0, device=dev)
    wt = torch.full((R, W + 2), np.nan if decay == 0 else 1.0, device=dev)[:, 1:1 + W]
    if decay:
        wt.copy_(torch.from_numpy(w))
    out = big[:R, 2:2 + W]
    out.copy_(torch.from_numpy(w))
    blse = torch.zeros((T, H + 3), device=dev)
    blse[:, 1:1 + H] = torch.from_numpy(lse)
    got = ops.accumulate_attention_weights(
        q, blse[:, 1:1 + H], torch.from_numpy(cache).to(dev), _i32(qsl, dev), _i32(seq, dev), _i32(table, dev), bs,
        out if place == "in" else wt, decay=decay, window_size=window, replay_start=_i32(rep, dev), base_offsets=_i32(off, dev),
        is_valid_token=None if ok is None else torch.from_numpy(ok).to(dev),
        sink=None if s is None else torch.from_numpy(s).to(dev), rope_dim=rope, out=None if place == "in" else out)
    assert got.data_ptr() == out.data_ptr()
    _close(out, want, tol, f"q {q_lens} prefix {prefix} H {H} D {D}")
    out.fill_(-3.0)
    assert bool((big == -3.0).all())  # nothing around the output is written


@pytest.mark.parametrize("q_lens,prefix,H,window", [
    ([1], [0], 1, 0), ([1], [31], 16, 0), ([1], [127], 16, 0), ([1], [128], 64, 0), ([1, 1, 1], [5, 300, 0], 64, 0), ([9], [0], 16, 0),
    ([130], [3], 8, 0), ([5, 0, 33], [200, 9, 1], 16, 128), ([4], [1000], 64, 128), ([3], [700], 128, 0),
    ([1, 1], [3000, 2000], 20, 0), ([40], [60], 4, 1), ([17, 2], [0, 90], 1, 33), ([21], [40], 70, 7), ([3], [150], 129, 0),
    ([2, 1], [80, 260], 300, 0), ([300], [0], 3, 0), ([0, 0, 4], [70, 0, 0], 24, 0)])
def test_shapes(cuda_device, q_lens, prefix, H, window):
    _run(cuda_device, sum(q_lens) + H, q_lens, prefix, H, window=window)


@pytest.mark.parametrize("D,rope", [(512, 0), (512, 128), (512, 448), (256, 64), (256, 0), (256, 192), (128, 64), (128, 0)])
@pytest.mark.parametrize("H", [5, 64])
def test_record_shapes(cuda_device, D, rope, H):
    _run(cuda_device, D + rope + H, [3, 7], [200, 133], H, D, rope)


@pytest.mark.parametrize("seed", range(30))
def test_fuzz(cuda_device, seed):
    rng = np.random.default_rng(700 + seed)
    R = int(rng.integers(1, 6))
    _run(cuda_device, seed, rng.integers(0, 30, size=R) + (np.arange(R) == 0), rng.integers(0, 400, size=R),
         H=int(rng.choice([1, 2, 5, 8, 16, 20, 32, 48, 64, 100, 140])), D=int(rng.choice([128, 256, 512])),
         rope=int(rng.choice([0, 64])), bs=int(rng.choice([1, 7, 16, 64])), window=int(rng.choice([0, 0, 1, 50, 300])),
         sink=bool(rng.integers(2)), replay=bool(rng.integers(2)), base=bool(rng.integers(2)), valid=bool(rng.integers(2)),
         missing=float(rng.choice([0.0, 0.2, 1.0])), pad=int(rng.choice([0, 3])), std=float(rng.choice([0.5, 6.0])),
         layout=str(rng.choice(["thd", "htd", "slice"])), decay=float(rng.choice([1.0, 0.0, 0.7])),
         place=str(rng.choice(["in", "out"])), narrow=int(rng.choice([0, 3, 200])))


def test_many_requests(cuda_device):
    """Neighbouring tokens of different requests; more of them than CTAs."""
    rng = np.random.default_rng(8)
    _run(cuda_device, 8, [1] * 300, rng.integers(0, 200, size=300), 16, 128, bs=16)
    _run(cuda_device, 9, rng.integers(0, 3, size=400), rng.integers(0, 90, size=400), 8, 128, bs=16, pad=1)
    _run(cuda_device, 10, [1] * 40, rng.integers(0, 500, size=40), 40, 512)


@pytest.mark.parametrize("q_lens,prefix,H,D,window", [
    ([64, 9, 0, 40], [3000, 1500, 5, 10], 16, 128, 0), ([50, 21], [2500, 40], 5, 256, 2000), ([70], [3], 128, 128, 0),
    ([200, 40], [300, 1800], 32, 128, 0), ([8] * 30, list(range(0, 2400, 80)), 8, 128, 1100), ([600], [0], 24, 128, 0)])
def test_rows_of_several_ctas(cuda_device, q_lens, prefix, H, D, window):
    """Rows whose columns are shared out over CTAs."""
    _run(cuda_device, H + D, q_lens, prefix, H, D, window=window, pad=3, missing=0.05)


@pytest.mark.parametrize("q_lens,prefix,H", [([1], [130000], 16), ([1, 1, 2], [60000, 3, 70000], 40), ([3], [110000], 129)])
def test_many_tiles_of_few_columns(cuda_device, q_lens, prefix, H):
    """CTAs with many tiles that share one column tile, or few."""
    _run(cuda_device, H, q_lens, prefix, H, 128)


def test_fewer_rows_than_new_tokens(cuda_device):
    """seq_lens below the query length: the first tokens lie before row 0."""
    _run(cuda_device, 1, [9, 20], [-4, -20], 6, 128, 0, bs=16)


@pytest.mark.parametrize("what", ["scale 247", "scale 255", "byte", "rope nan", "rope inf"])
def test_non_finite_rows(cuda_device, what):
    """Every way a record can hold a NaN or an infinity: its own weight alone notices."""
    d, rng = cuda_device, np.random.default_rng(13)
    D, bs, bad, n, H = 256, 16, 53, 75, 20
    cache = _cache(rng, 8, bs, D, 64)
    clean = cache.copy()
    page, at = cache[bad // bs], bad % bs
    scales = page[bs * (D + 64) + at * (D // 64):]
    if what.startswith("scale"):
        page[at * (D + 64) + 3] = 0xFE
        scales[0] = int(what.split()[1])
    elif what == "byte":
        page[at * (D + 64) + 130] = 0xFF
    else:
        page[at * (D + 64) + D - 64 + 6:at * (D + 64) + D - 64 + 8] = (0xC1, 0x7F) if what == "rope nan" else (0x80, 0xFF)
    q, q64 = _query(rng, 10, H, D, 1.0, d, "thd")
    lse = np.full((10, H), 5.0, np.float32)
    table = np.arange(8, dtype=np.int32)[None, :]
    w = rng.random((1, n)).astype(np.float32)
    res = []
    for c in (cache, clean):
        wt = torch.from_numpy(w).to(d)
        res.append(ops.accumulate_attention_weights(q, torch.from_numpy(lse).to(d), torch.from_numpy(c).to(d), _i32([0, 10], d),
                                                    _i32([n], d), _i32(table, d), bs, wt).cpu())
    keep = torch.arange(n) != bad
    assert torch.equal(res[0][:, keep], res[1][:, keep])
    want, tol = plain.accumulate(q64, lse, clean, [0, 10], [n], table, bs, 64, np.float64(np.float32(D ** -0.5)), w)
    _close(res[1], want, tol)
    if what != "scale 247":
        assert not bool(torch.isfinite(res[0][0, bad]))


def test_non_finite_queries_and_logs(cuda_device):
    """A NaN in a query or an lse reaches what its token sees; a token that sees nothing none."""
    d, rng = cuda_device, np.random.default_rng(14)
    cache = torch.from_numpy(_cache(rng, 4, 64, 512, 64)).to(d)
    q, _ = _query(rng, 6, 10, 512, 1.0, d, "thd")
    lse = torch.full((6, 10), 6.0, device=d)
    args = (cache, _i32([0, 6], d), _i32([200], d), _i32(np.arange(4)[None, :], d), 64)
    base = ops.accumulate_attention_weights(q, lse, *args, torch.zeros(1, 200, device=d))
    assert bool(torch.isfinite(base).all())
    bad = q.clone()
    bad[2, 3, 77] = float("nan")
    got = ops.accumulate_attention_weights(bad, lse, *args, torch.zeros(1, 200, device=d))
    assert bool(torch.isnan(got[0, :197]).all()) and torch.equal(got[0, 197:], base[0, 197:])
    for value in (float("nan"), -float("inf")):
        worse = lse.clone()
        worse[2, 3] = value
        got = ops.accumulate_attention_weights(q, worse, *args, torch.zeros(1, 200, device=d))
        assert bool(torch.isnan(got[0, :197]).all()) == (value != value) and torch.equal(got[0, 197:], base[0, 197:])
        # padding tokens have no influence, whatever they hold
        valid = torch.ones(6, dtype=torch.bool, device=d)
        valid[2] = False
        a = ops.accumulate_attention_weights(bad, worse, *args, torch.zeros(1, 200, device=d), is_valid_token=valid)
        b = ops.accumulate_attention_weights(q, lse, *args, torch.zeros(1, 200, device=d), is_valid_token=valid)
        assert torch.equal(a, b)
    # all of a token's weight on the sink
    got = ops.accumulate_attention_weights(q, lse, *args, torch.zeros(1, 200, device=d), sink=torch.full((10,), float("inf"), device=d))
    assert bool((got == 0).all())
    got = ops.accumulate_attention_weights(q, lse, *args, torch.zeros(1, 200, device=d), sink=torch.full((10,), -float("inf"), device=d))
    assert torch.equal(got, base)


def test_weights_of_an_attention_call_sum_to_one(cuda_device):
    """With the attention's own lse and no sink every (token, head) hands out 1 in all."""
    d, rng = cuda_device, np.random.default_rng(15)
    H, n, new = 40, 1500, 30
    host = _cache(rng, 24, 64, 512, 64)
    cache = torch.from_numpy(host).to(d)
    q, q64 = _query(rng, new, H, 512, 2.0, d, "thd")
    meta = (_i32([0, new], d), _i32([n], d))
    table = _i32(rng.permutation(24)[None, :], d)
    _, lse = ops.chunk_mla_attention(q, cache, *meta, _i32(np.zeros(new), d), table, 64)
    w = ops.accumulate_attention_weights(q, lse, cache, *meta, table, 64, torch.zeros(1, n, device=d))
    # a score is off by at most D 2^-23 scale sum|q k| in either call, and lse by as much again
    k = np.abs(rows_of(host, 64, 512, 64, np.arange(24 * 64)))
    ds = 512 * 2.0 ** -23 * 512 ** -0.5 * float((np.abs(q64).reshape(-1, 512) @ k.T).max())
    assert abs(float(w.double().sum()) / (new * H) - 1.0) <= 3 * ds
    # later rows are seen by fewer tokens: the last row by the last token alone
    assert float(w[0, n - 1]) <= H


def test_same_bits_again_and_in_any_batch(cuda_device):
    d, rng = cuda_device, np.random.default_rng(16)
    cache = torch.from_numpy(_cache(rng, 40, 64, 512, 64)).to(d)
    q, _ = _query(rng, 90, 48, 512, 2.0, d, "thd")
    lse = torch.full((90, 48), 6.0, device=d)
    args = (q, lse, cache, _i32([0, 90], d), _i32([2500], d), _i32(rng.permutation(40)[None, :], d), 64)
    one = ops.accumulate_attention_weights(*args, torch.zeros(1, 2500, device=d))
    for _ in range(5):
        assert torch.equal(ops.accumulate_attention_weights(*args, torch.zeros(1, 2500, device=d)), one)


def test_captured_on_another_stream_and_beside_another(cuda_device):
    d, rng = cuda_device, np.random.default_rng(17)
    cases = []
    for T, H, n in ((64, 64, 900), (1, 16, 2000)):
        cache = torch.from_numpy(_cache(rng, 40, 64, 512, 64)).to(d)
        q, _ = _query(rng, T, H, 512, 2.0, d, "thd")
        cases.append((q, torch.full((T, H), 6.0, device=d), cache, _i32([0, T], d), _i32([n], d),
                      _i32(rng.permutation(40)[None, :], d), 64, torch.rand((1, n), device=d)))
    run = lambda c, out: ops.accumulate_attention_weights(*c, decay=0.5, out=out)  # noqa: E731
    want = [run(c, torch.zeros_like(c[-1])) for c in cases]
    torch.cuda.synchronize(d)
    graphs, outs = [], [torch.zeros_like(c[-1]) for c in cases]
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, o)
        graphs.append(g)
    streams = [torch.cuda.Stream(d), torch.cuda.Stream(d)]
    for _ in range(3):
        for s, g, o in zip(streams, graphs, outs):
            o.zero_()
            s.wait_stream(torch.cuda.current_stream(d))
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize(d)
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_far_pages(cuda_device):
    """Records past byte 2^32 of a cache, odd page size."""
    d, rng = cuda_device, np.random.default_rng(18)
    bs, stride = 3, 1760
    pages = (1 << 32) // stride + 900
    cache = torch.zeros((pages, stride), dtype=torch.uint8, device=d)
    few = _cache(rng, 60, bs, 512, 64)
    where = np.sort(rng.choice(np.arange(pages - 800, pages), size=60, replace=False))
    cache[torch.from_numpy(where).to(d), :few.shape[1]] = torch.from_numpy(few).to(d)
    q, q64 = _query(rng, 3, 20, 512, 1.0, d, "thd")
    lse = np.full((3, 20), 5.0, np.float32)
    w = np.zeros((1, 170), np.float32)
    got = ops.accumulate_attention_weights(q, torch.from_numpy(lse).to(d), cache, _i32([0, 3], d), _i32([170], d), _i32(where[None, :], d),
                                           bs, torch.from_numpy(w).to(d))
    want, tol = plain.accumulate(q64, lse, few, [0, 3], [170], np.arange(60)[None, :], bs, 64, np.float64(np.float32(512 ** -0.5)), w)
    _close(got, want, tol)


def test_no_tokens(cuda_device):
    """Nothing new: the weights fade all the same."""
    d = cuda_device
    cache, w = torch.zeros((2, 64 * 584), dtype=torch.uint8, device=d), torch.ones(2, 100, device=d)
    out = ops.accumulate_attention_weights(torch.zeros((0, 8, 512), dtype=BF16, device=d), torch.zeros((0, 8), device=d), cache,
                                           _i32([0, 0, 0], d), _i32([70, 0], d), _i32([[0, 1], [0, 1]], d), 64, w, decay=0.5)
    assert bool((out[0, :70] == 0.5).all()) and bool((out[0, 70:] == 1).all()) and bool((out[1] == 1).all())


def test_refusals(cuda_device):
    d = cuda_device
    q, lse = torch.zeros((2, 4, 512), dtype=BF16, device=d), torch.zeros((2, 4), device=d)
    cache, n = torch.zeros((2, 64 * 584), dtype=torch.uint8, device=d), torch.zeros(3, dtype=I32, device=d)
    table, w = torch.zeros((2, 2), dtype=I32, device=d), torch.zeros(2, 100, device=d)

    def call(q=q, lse=lse, qsl=n, seq=n[:2], table=table, w=w, **kw):
        return ops.accumulate_attention_weights(q, lse, cache, qsl, seq, table, 64, w, **kw)
    call()
    for kw, kind, text in [
            (dict(q=q.float()), TypeError, "q must"), (dict(lse=lse.double()), TypeError, "lse must"),
            (dict(lse=lse[:1]), ValueError, "lse must"), (dict(qsl=n[:2]), ValueError, "query_start_loc"),
            (dict(table=table[:1]), ValueError, "block_table"), (dict(w=w[:1]), ValueError, "at least"),
            (dict(w=w.double()), TypeError, "weights"), (dict(w=w[:1].expand(2, 100)), ValueError, "overlap"),
            (dict(out=w[:, :50]), ValueError, "at least"), (dict(sink=lse[0, :3]), ValueError, "sink"),
            (dict(q=q[:, :1].expand(2, 4, 512)), ops.PskError, "strides"), (dict(decay=-1.0), ops.PskError, "decay"),
            (dict(workspace=torch.zeros(0, dtype=torch.uint8, device=d)), ops.PskError, "workspace")]:
        if text == "workspace" and ops.accumulate_attention_weights_workspace_bytes(d) == 0:
            continue
        with pytest.raises(kind, match=text):
            call(**kw)


def test_strides_of_single_tokens_and_heads(cuda_device):
    """A size-1 dim may carry any stride, 0 from broadcasting among them."""
    d, rng = cuda_device, np.random.default_rng(19)
    cache = torch.from_numpy(_cache(rng, 4, 64, 128, 64)).to(d)
    meta = (_i32([0, 1], d), _i32([200], d), _i32(np.arange(4)[None, :], d), 64)
    for H in (1, 5):
        q, _ = _query(rng, 1, H, 128, 1.0, d, "thd")
        want = ops.accumulate_attention_weights(q, torch.full((1, H), 5.0, device=d), cache, *meta, torch.zeros(1, 200, device=d))
        for view in (q.as_strided((1, H, 128), (0, 128, 1)), q.as_strided((1, H, 128), (8, 128 if H > 1 else 0, 1))):
            got = ops.accumulate_attention_weights(view, torch.full((1, H), 5.0, device=d), cache, *meta, torch.zeros(1, 200, device=d))
            assert torch.equal(got, want)


def test_more_requests_than_a_warp_plans(cuda_device):
    """The range of a CTA found by one warp (up to 128 requests) and by all of them."""
    rng = np.random.default_rng(20)
    for R in (32, 33, 128, 129, 1000):
        _run(cuda_device, R, rng.integers(0, 4, size=R) + (np.arange(R) == 0), rng.integers(0, 150, size=R), 6, 128, bs=16)
