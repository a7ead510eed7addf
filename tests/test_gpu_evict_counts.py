"""Moves of cache rows: lists and counts at the ends of their range."""
import numpy as np
import pytest
import torch

from oracle import evict as plain
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _cache(rng, pages, dev):
    host = rng.integers(0, 256, (pages, 16 * 68), dtype=np.uint8)
    return host, torch.from_numpy(host).to(dev)


@pytest.mark.parametrize("room", [2**31 - 1, 2**31 - 32, 2**31 - 33])
def test_room_for_the_most_moves(cuda_device, room):
    d, rng = cuda_device, np.random.default_rng(1)
    host, cache = _cache(rng, 8, d)
    moves = torch.empty((1, room, 2), dtype=I32, device=d)  # 17 GB, of which the first entries count
    few = np.stack([np.arange(70, 110), np.arange(40)], 1)
    moves[0, :40] = torch.from_numpy(few.astype(np.int32)).to(d)
    table = np.arange(8)[None, ::-1].copy()
    ops.move_cache_rows(cache, torch.from_numpy(table.astype(np.int32)).to(d), moves, torch.tensor([40], dtype=I32, device=d), 16, 128,
                        record=ops.PSK_REC_MXFP4)
    want, _ = plain.move(host, 16, 64, 4, table, [few], [40])
    assert np.array_equal(cache.cpu().numpy(), want)


def test_counts_below_zero(cuda_device):
    """The least count of all, from which the moves before a tile cannot be taken off."""
    d, rng = cuda_device, np.random.default_rng(2)
    host, cache = _cache(rng, 32, d)
    table = np.arange(32).reshape(4, 8)
    moves = np.stack([np.tile(np.arange(64, 128), (4, 1)), np.tile(np.arange(64), (4, 1))], 2)
    counts = [-2**31, -1, 64, 3 - 2**31]
    ops.move_cache_rows(cache, torch.from_numpy(table.astype(np.int32)).to(d), torch.from_numpy(moves.astype(np.int32)).to(d),
                        torch.tensor(counts, dtype=I32, device=d), 16, 128, record=ops.PSK_REC_MXFP4)
    want, _ = plain.move(host, 16, 64, 4, table, moves, counts)
    assert np.array_equal(cache.cpu().numpy(), want)
