"""Attention with equal weights, where every row counts: queries of zero and no sink
give lse = log(number of visible rows) and out = the rows' mean.

Row j holds a single 1, in dim j mod D, so out[d] is the number of visible rows of that
kind over the number of all.  Weights of 1 and their sums below 2^24 are exact in binary32.
What is left in lse is log2 (within a step, 2^-23 relative), log 2 and one product (half a
step each): 2^-22; in out a reciprocal and one product (2^-23) and the rounding to bf16
(2^-8).  One row more or less changes lse by 1 / count, far beyond that."""
import numpy as np
import pytest
import torch

import oracle
from oracle import attention as plain
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu

BS = 64


@pytest.fixture(autouse=True)
def no_wait_expires(cuda_device):
    before = ops.device_wait_timeouts()
    yield
    torch.cuda.synchronize()
    assert ops.device_wait_timeouts() == before


def _unit_rows(slots, D):
    """A cache of `slots` rows (a multiple of the page size), row j with a 1 in dim j mod D."""
    rows = np.zeros((slots, D), np.uint16)
    rows[np.arange(slots), np.arange(slots) % D] = 0x3F80
    stride = -(-BS * oracle.fp8_record_bytes(D, 64) // 16) * 16
    cache = np.zeros((slots // BS, stride), np.uint8)
    oracle.quantize_and_insert_k_cache(rows, np.arange(slots), cache, BS, D, 64)
    return cache


def _check(out, lse, visible, D, what):
    """`visible`: the visible slots of each token, with repetitions."""
    T, H = lse.shape
    n = np.array([len(v) for v in visible], np.float64)
    kinds = np.stack([np.bincount(np.asarray(v, np.int64) % D, minlength=D) for v in visible])
    with np.errstate(divide="ignore"):
        want = np.log(n)[:, None].repeat(H, 1)
    got = lse.double().cpu().numpy()
    none = n == 0
    assert (got[none] == -np.inf).all(), what
    off = np.abs(got[~none] - want[~none])
    assert (off <= np.abs(want[~none]) * 2.0 ** -22).all(), f"{what}: counts {np.exp(got[~none])[off.argmax() // H]}"
    mean = kinds / np.maximum(n, 1)[:, None]
    err = np.abs(out.double().cpu().numpy() - mean[:, None, :])
    assert (err <= mean[:, None, :] * (2.0 ** -8 + 2.0 ** -23) * (1 + 2.0 ** -8)).all(), what


def _i32(a, d):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(d)


@pytest.mark.parametrize("T,H,D,C,split", [
    (1, 16, 512, 640, 128), (1, 1, 128, 3, 1), (64, 64, 512, 640, 128), (9, 64, 512, 129, 129), (5, 24, 256, 2000, 7),
    (2, 128, 512, 2300, 200), (160, 9, 128, 700, 300), (40, 130, 256, 515, 0), (1, 64, 512, 20000, 9000), (400, 3, 128, 90, 40)])
def test_sparse_counts(cuda_device, T, H, D, C, split):
    d = cuda_device
    rng = np.random.default_rng(T + H + C)
    a, b = _unit_rows(4096, D), _unit_rows(8192, D)
    idx = np.concatenate([rng.integers(0, 4096, size=(T, split)), rng.integers(0, 8192, size=(T, C - split))], 1)
    idx[rng.random((T, C)) < 0.1] = -1
    idx[:, C // 3] = 1 << 20
    if T > 4:
        idx[3] = -1
        idx[4, 1:] = -1
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device=d)
    out, lse = ops.sparse_mla_attention(q, torch.from_numpy(a).to(d), _i32(idx, d), BS, extra_cache=torch.from_numpy(b).to(d),
                                        extra_block_size=BS, split=split)
    cap = np.where(np.arange(C) < split, 4096, 8192)
    _check(out, lse, [r[(r >= 0) & (r < cap)] for r in idx], D, f"T {T} H {H} C {C}")


def _chunk(d, q_lens, seq, H, D, window, width, seed, missing=0.0):
    """A call over a table of `width` columns, of which a request uses the first; the
    columns past its length name pages like any other."""
    rng = np.random.default_rng(seed)
    q_lens, seq = np.asarray(q_lens), np.asarray(seq)
    R, T = len(seq), int(q_lens.sum())
    pages = 4096 // BS * 2
    cache = _unit_rows(pages * BS, D)
    table = rng.integers(0, pages, size=(R, width))
    table[rng.random((R, width)) < missing] = -1
    qsl = np.concatenate([[0], np.cumsum(q_lens)])
    t2r = np.repeat(np.arange(R), q_lens)
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device=d)
    out, lse = ops.chunk_mla_attention(q, torch.from_numpy(cache).to(d), _i32(qsl, d), _i32(seq, d), _i32(t2r, d),
                                       _i32(table, d), BS, window_size=window)
    seen = [plain.visible_slots(t, qsl, seq, t2r, table, BS, pages, window) for t in range(T)]
    _check(out, lse, seen, D, f"q {q_lens[:5]} seq {seq[:5]} H {H} window {window} width {width}")


@pytest.mark.parametrize("q_lens,seq,H,D,window", [
    ([1], [1], 1, 512, 0), ([1, 1], [9000, 20000], 64, 512, 0), ([70, 3], [900, 130], 16, 512, 0), ([40], [700], 3, 128, 128),
    ([33, 31], [500, 40], 130, 256, 200), ([5, 0, 9], [1000, 10, 9], 32, 128, 0)])
def test_chunk_counts(cuda_device, q_lens, seq, H, D, window):
    _chunk(cuda_device, q_lens, seq, H, D, window, -(-max(seq) // BS), sum(q_lens) + H, missing=0.05)


@pytest.mark.parametrize("q_lens,seq,H,D", [
    ([1] * 64, [1024 - i for i in range(64)], 64, 512), ([1], [128], 64, 512), ([1] * 256, [1 + 2 * i for i in range(256)], 64, 128),
    ([1, 1], [300, 1], 16, 512), ([40, 3, 1], [60, 400, 1], 8, 512), ([9] * 7, [9 + 30 * i for i in range(7)], 33, 256)])
@pytest.mark.parametrize("window", [0, 128])
def test_chunk_wide_tables(cuda_device, q_lens, seq, H, D, window):
    """Tables for 131072 positions over short contexts: more parts than tiles, most of them empty."""
    _chunk(cuda_device, q_lens, seq, H, D, window, 131072 // BS, len(seq) + H)




def test_chunk_narrowed_table(cuda_device):
    """The first columns of a wide table: the plan, the scratch and the bits of a tight one."""
    d, R, H, W = cuda_device, 64, 64, 16
    cache = torch.from_numpy(_unit_rows(4096, 512)).to(d)
    wide = torch.randint(0, 4096 // BS, (R, 2048), dtype=torch.int32, device=d)
    q = torch.randn((R, H, 512), device=d).to(torch.bfloat16)
    cu, seq, t2r = (torch.arange(R + 1, dtype=torch.int32, device=d), torch.arange(1, R + 1, dtype=torch.int32, device=d) * 16,
                    torch.arange(R, dtype=torch.int32, device=d))
    need = [ops.chunk_mla_attention_workspace_bytes(d, R, R, H, 512, w, BS) for w in (W, 2048)]
    assert need[0] < need[1]
    ws = torch.empty((max(need[0], 16),), dtype=torch.uint8, device=d)
    a = ops.chunk_mla_attention(q, cache, cu, seq, t2r, wide[:, :W], BS, workspace=ws)
    b = ops.chunk_mla_attention(q, cache, cu, seq, t2r, wide[:, :W].contiguous(), BS)
    c = ops.chunk_mla_attention(q, cache, cu, seq, t2r, wide, BS)
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y)
        # other parts: the same weights, rounded to bf16 against other references
        assert torch.allclose(x.float(), z.float(), rtol=2**-6, atol=2**-8)
