"""GPU parity of the batch-metadata kernels with their plain forms (exact)."""
import numpy as np
import pytest
import torch

from oracle import batch_meta
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu


def _i32(a, dev):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def _ragged(rng, R, T):
    """Query lengths of R requests that sum to T, empty ones among them."""
    return np.bincount(rng.integers(0, R, size=T), minlength=R)


def _check_slots(d, rng, R, T, pad, bs, cbs, ratio, comp, with_base, context=300):
    q = _ragged(rng, R, T)
    seq = (q + rng.integers(0, context, size=R)).astype(np.int32)
    if R > 2:
        seq[1] = max(int(q[1]) - 2, 0)  # more new tokens than positions: the first lie before 0
    qsl = np.concatenate([[0], np.cumsum(q)])
    width = int(rng.integers(1, int(seq.max()) // bs + 3))
    table = rng.integers(-1, 1 << 30, size=(R, width)).astype(np.int32)
    ctable = rng.integers(-1, 50, size=(R, max(1, width // ratio))).astype(np.int32) if comp else None
    base = rng.integers(0, 2, size=R) if with_base else None
    cbase = rng.integers(0, 2, size=R) if with_base else None
    want = batch_meta.compute_slot_mappings(qsl, seq, table, bs, T + pad, base, ctable, cbs, cbase,
                                            ratio)
    got = ops.compute_slot_mappings(_i32(qsl, d), _i32(seq, d), _i32(table, d), bs, T + pad,
                                    base_offsets=_i32(base, d), compressed_block_table=_i32(ctable, d),
                                    compressed_block_size=cbs, compressed_base_offsets=_i32(cbase, d),
                                    compress_ratio=ratio)
    for name, g, w in zip(("positions", "token_to_req", "slots", "compressed slots"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("seed", range(24))
def test_slot_mappings_fuzz(cuda_device, seed):
    rng = np.random.default_rng(7000 + seed)
    _check_slots(cuda_device, rng, R=int(rng.integers(1, 40)), T=int(rng.integers(0, 900)),
                 pad=int(rng.choice([0, 1, 130])), bs=int(rng.choice([1, 3, 16, 64])),
                 cbs=int(rng.choice([1, 5, 64])), ratio=int(rng.choice([1, 3, 4, 128])),
                 comp=bool(rng.integers(0, 2)), with_base=bool(rng.integers(0, 2)))


@pytest.mark.parametrize("R,T", [(1, 1), (5000, 7001), (9, 170003), (4095, 3), (4096, 3),
                                 (9, 250003), (5000, 240001), (3, 233471), (3, 233472)])
def test_slot_mappings_sizes(cuda_device, R, T):
    """One token; more requests than are staged in shared memory (and the last
    that are); enough tokens for four per thread with a ragged end."""
    rng = np.random.default_rng(R + T)
    _check_slots(cuda_device, rng, R, T, pad=3, bs=64, cbs=64, ratio=4, comp=True, with_base=False)


def test_slot_mappings_partial_outputs_and_bounds(cuda_device):
    """Outputs left out, an output that is not 16-byte aligned (one per thread is
    stored), and entries around the outputs that stay as they were."""
    for T in (200001, 250001):
        _check_partial(cuda_device, T)


def _check_partial(d, T):
    R = 3
    rng = np.random.default_rng(5)
    q = _ragged(rng, R, T)
    seq = (q + 17).astype(np.int32)
    qsl = np.concatenate([[0], np.cumsum(q)])
    table = rng.integers(0, 1000, size=(R, int(seq.max()) // 64 + 1)).astype(np.int32)
    want = batch_meta.compute_slot_mappings(qsl, seq, table, 64, T)
    for shift in (0, 1):
        buf = torch.full((T + 8,), -77, dtype=torch.int64, device=d)
        out = buf[4 + shift:4 + shift + T]
        ops.compute_slot_mappings(_i32(qsl, d), _i32(seq, d), _i32(table, d), 64, T, slot_mapping=out)
        assert np.array_equal(out.cpu().numpy(), want[2])
        rest = torch.cat([buf[:4 + shift], buf[4 + shift + T:]])
        assert bool((rest == -77).all())


def test_slot_mappings_past_int32(cuda_device):
    """Slots past 2^31 stay exact (pages near INT32_MAX, pages of 64)."""
    d = cuda_device
    table = np.array([[2**31 - 1, 2**31 - 2]], np.int32)
    want = batch_meta.compute_slot_mappings([0, 100], [100], table, 64, 100)
    got = ops.compute_slot_mappings(_i32([0, 100], d), _i32([100], d), _i32(table, d), 64, 100)
    assert int(want[2].max()) > 2**36
    assert np.array_equal(got[2].cpu().numpy(), want[2])


def _check_extend(d, rng, R, width, pool_size, held, bs, ratio, head, extra=0, most=None):
    seq = rng.integers(-2, (most or width) * bs * ratio + bs, size=R).astype(np.int32)
    counts = rng.integers(-1, width + 2, size=R).astype(np.int32) if held else None
    pool = rng.permutation(1 << 20)[:pool_size].astype(np.int32)
    big = rng.integers(-9, 9, size=(R, width + extra)).astype(np.int32)
    table = big[:, extra // 2:extra // 2 + width]
    want, wc, wh, we = batch_meta.extend_block_tables(seq, pool, table, bs, counts,
                                                      0 if head is None else head, ratio)
    g_big = _i32(big, d)
    g_table = g_big[:, extra // 2:extra // 2 + width]
    err = torch.full((1,), 5, dtype=torch.int32, device=d)
    args = (_i32(seq, d), _i32(pool, d), g_table, bs)
    kw = dict(page_counts=_i32(counts, d), pool_head=None if head is None else _i32([head], d),
              compress_ratio=ratio, err_count=err)
    for _ in range(2):  # a repeated call gives the same result
        _, gc, gh = ops.extend_block_tables(*args, **kw)
        assert np.array_equal(g_table.cpu().numpy(), want)
        assert np.array_equal(gc.cpu().numpy(), wc)
        assert int(gh) == wh
    assert int(err) == 5 + 2 * we
    rest = np.delete(g_big.cpu().numpy(), np.s_[extra // 2:extra // 2 + width], axis=1)
    assert np.array_equal(rest, np.delete(big, np.s_[extra // 2:extra // 2 + width], axis=1))


@pytest.mark.parametrize("seed", range(24))
def test_extend_fuzz(cuda_device, seed):
    rng = np.random.default_rng(8000 + seed)
    R, width = int(rng.integers(1, 300)), int(rng.integers(0, 70))
    _check_extend(cuda_device, rng, R, width, pool_size=int(rng.integers(0, R * width + 20)),
                  held=bool(rng.integers(0, 2)), bs=int(rng.choice([1, 3, 16, 64])),
                  ratio=int(rng.choice([1, 4, 7])), head=rng.choice([None, 0, -3, 11, 10**6]),
                  extra=int(rng.choice([0, 1, 3, 6])))


@pytest.mark.parametrize("R,width", [(5001, 5), (1, 4099), (1217, 33)])
def test_extend_many_rows(cuda_device, R, width):
    """Several rows per CTA, one very wide row; a pool that runs out half-way."""
    rng = np.random.default_rng(R)
    for pool in (R * width + 1, R * width // 3):
        _check_extend(cuda_device, rng, R, width, pool, True, 16, 1, 2)


def test_extend_without_rows(cuda_device):
    d = cuda_device
    z = torch.zeros((0,), dtype=torch.int32, device=d)
    _, counts, head = ops.extend_block_tables(z, torch.arange(4, dtype=torch.int32, device=d),
                                              torch.zeros((0, 3), dtype=torch.int32, device=d), 16,
                                              pool_head=_i32([3], d))
    assert counts.shape == (0,) and int(head) == 3


def test_batch_meta_captured_on_a_side_stream(cuda_device):
    """Grow the tables, then map slots, captured once and replayed on new lengths."""
    d = cuda_device
    R, width, bs, T = 6, 20, 16, 40
    rng = np.random.default_rng(3)
    pool = rng.permutation(200).astype(np.int32)
    g_pool, seq = _i32(pool, d), torch.zeros(R, dtype=torch.int32, device=d)
    qsl = torch.zeros(R + 1, dtype=torch.int32, device=d)
    table = torch.zeros((R, width), dtype=torch.int32, device=d)
    outs = {}

    def step():
        ops.extend_block_tables(seq, g_pool, table, bs)
        outs["maps"] = ops.compute_slot_mappings(qsl, seq, table, bs, T)
    side = torch.cuda.Stream(d)
    side.wait_stream(torch.cuda.current_stream(d))
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize(d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        q = _ragged(rng, R, T - 4)
        lens = (q + rng.integers(0, 200, size=R)).astype(np.int32)
        cu = np.concatenate([[0], np.cumsum(q)])
        seq.copy_(_i32(lens, d))
        qsl.copy_(_i32(cu, d))
        graph.replay()
        want_t, _, _, _ = batch_meta.extend_block_tables(lens, pool, np.zeros((R, width), np.int32), bs)
        want = batch_meta.compute_slot_mappings(cu, lens, want_t, bs, T)
        assert np.array_equal(table.cpu().numpy(), want_t)
        for g, w in zip(outs["maps"], want):
            assert np.array_equal(g.cpu().numpy(), w)


def test_batch_meta_refusals(cuda_device):
    d = cuda_device
    seq, qsl = _i32([3], d), _i32([0, 3], d)
    table = _i32([[0, 1]], d)
    with pytest.raises(TypeError):
        ops.compute_slot_mappings(qsl.long(), seq, table, 16, 3)
    with pytest.raises(ValueError):
        ops.compute_slot_mappings(qsl[:1], seq, table, 16, 3)  # no end of the last request
    with pytest.raises(ValueError):
        ops.compute_slot_mappings(qsl, seq, table[:0], 16, 3)
    with pytest.raises(ValueError):
        ops.compute_slot_mappings(qsl, seq, table, 16, 3, slot_mapping=torch.zeros(2, dtype=torch.int64, device=d))
    with pytest.raises(ValueError):
        ops.compute_slot_mappings(qsl.cpu(), seq, table, 16, 3)
    with pytest.raises(ops.PskError):
        ops.compute_slot_mappings(qsl, seq, table, 0, 3)
    pool = _i32([4, 5], d)
    with pytest.raises(ops.PskError):  # the counts are read by every CTA: not updated in place
        ops.extend_block_tables(seq, pool, table, 16, page_counts=seq.clone(), page_counts_out=seq)
    with pytest.raises(ValueError):
        ops.extend_block_tables(_i32([1, 2], d), pool, table.expand(2, 2), 16)
