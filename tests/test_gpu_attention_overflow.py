"""Scores past the range of binary32: +infinity makes a (token, head) NaN, -infinity is a
weight of 0, and other heads and tokens are as without them, in every way the work is split."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu

BS = 64
SCALE = 1e38


def _cache(n, at, D, d):
    """n rows of zeros (rounded up to whole pages), but for row `at`, whose first dim is 1."""
    rows = np.zeros((-(-n // BS) * BS, D), np.uint16)
    rows[at, 0] = 0x3F80
    stride = -(-BS * oracle.fp8_record_bytes(D, 64) // 16) * 16
    cache = np.zeros((len(rows) // BS, stride), np.uint8)
    oracle.quantize_and_insert_k_cache(rows, np.arange(len(rows)), cache, BS, D, 64)
    return torch.from_numpy(cache).to(d)


def _query(T, H, D, d):
    """Heads 0, 1, 2, 0, 1, 2 ...: scores of 0 alone; +infinity at the row; -infinity there."""
    q = torch.zeros((T, H, D))
    q[:, 1::3, 0], q[:, 2::3, 0] = 16.0, -16.0
    return q.to(torch.bfloat16).to(d)


def _check(out, lse, seen, has):
    """`seen` rows of a token, of which the high one is one where `has`."""
    out, lse = out.double().cpu(), lse.double().cpu()
    for t in range(len(seen)):
        n, hit = seen[t], has[t]
        assert torch.allclose(lse[t, 0::3], torch.tensor(math.log(n), dtype=torch.float64), rtol=2**-22, atol=0)
        want = 1.0 / n if hit else 0.0
        assert bool(((out[t, 0::3, 0] - want).abs() <= want * 2**-8 * 1.01).all())
        assert bool((out[t, 0::3, 1:] == 0).all())
        if hit:
            assert bool(torch.isnan(out[t, 1::3]).all()) and bool(torch.isnan(lse[t, 1::3]).all())
        else:
            assert bool((out[t, 1::3] == 0).all())
            assert torch.allclose(lse[t, 1::3], torch.tensor(math.log(n), dtype=torch.float64), rtol=2**-22, atol=0)
        left = n - hit
        low = torch.tensor(math.log(left) if left else -math.inf, dtype=torch.float64)
        assert torch.allclose(lse[t, 2::3], low, rtol=2**-22, atol=0)
        assert bool((out[t, 2::3] == 0).all())


@pytest.mark.parametrize("T,H,D,n,at", [
    (1, 3, 128, 1, 0), (1, 3, 128, 128, 5), (1, 3, 128, 300, 200), (1, 16, 512, 640, 639), (64, 64, 512, 640, 100),
    (2, 6, 128, 5000, 10), (2, 6, 128, 5000, 4990), (160, 5, 256, 400, 390), (3, 70, 512, 129, 128)])
@pytest.mark.parametrize("sink", [False, True])
def test_sparse(cuda_device, T, H, D, n, at, sink):
    d = cuda_device
    idx = torch.arange(n, dtype=torch.int32, device=d)[None].repeat(T, 1)
    s = torch.full((H,), -1e30, device=d) if sink else None  # a share of 0
    out, lse = ops.sparse_mla_attention(_query(T, H, D, d), _cache(n, at, D, d), idx, BS, softmax_scale=SCALE, sink=s)
    _check(out, lse, [n] * T, [True] * T)


@pytest.mark.parametrize("T,H,D,n,at", [
    (1, 3, 128, 1, 0), (1, 64, 512, 700, 3), (40, 3, 128, 300, 280), (12, 16, 512, 200, 150), (5, 33, 256, 129, 0)])
def test_chunk(cuda_device, T, H, D, n, at):
    """Tokens at the last T positions, some of which lie before the row."""
    d = cuda_device
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=d)  # noqa: E731
    cache = _cache(n, at, D, d)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device=d)[None]
    out, lse = ops.chunk_mla_attention(_query(T, H, D, d), cache, i32([0, T]), i32([n]), i32([0] * T), table, BS,
                                       softmax_scale=SCALE)
    pos = range(n - T, n)
    _check(out, lse, [p + 1 for p in pos], [p >= at for p in pos])
