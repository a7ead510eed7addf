"""Attention weights of a request by itself and among others, and of a call that holds fewer tokens
than its metadata names."""
import numpy as np
import pytest
import torch

from oracle import attn_weights as plain
from paged_sparse_kv_gb300 import ops
from test_gpu_attn_weights import _cache, _close, _i32, _lse, _query, no_wait_expires  # noqa: F401

pytestmark = pytest.mark.gpu
BS, SCALE = 16, np.float64(np.float32(128 ** -0.5))


def _inputs(dev, seed, q_lens, prefix, H):
    rng = np.random.default_rng(seed)
    seq, qsl = np.array(q_lens) + np.array(prefix), np.concatenate([[0], np.cumsum(q_lens)])
    R, width = len(seq), -(-int(seq.max()) // BS)
    table = rng.permutation(R * width).reshape(R, width).astype(np.int32)
    cache = _cache(rng, R * width, BS, 128, 64)
    q, q64 = _query(rng, int(qsl[-1]), H, 128, 1.5, dev, "thd")
    lse = _lse(q64, cache, BS, 64, table, seq, qsl, None, SCALE, rng)
    return q, q64, lse, cache, qsl, seq, table, rng.random((R, int(seq.max()))).astype(np.float32)


def _run(dev, q, lse, cache, qsl, seq, table, w):
    out = torch.from_numpy(w).to(dev)
    return ops.accumulate_attention_weights(q, torch.from_numpy(lse).to(dev), torch.from_numpy(cache).to(dev), _i32(qsl, dev),
                                            _i32(seq, dev), _i32(table, dev), BS, out)


@pytest.mark.parametrize("q_lens,prefix,H", [([3, 1, 40, 7], [900, 30, 200, 2500], 8), ([1] * 20, list(range(0, 2000, 100)), 16),
                                             ([200, 2, 1], [100, 1500, 3000], 64)])
def test_alone_and_in_a_batch(cuda_device, q_lens, prefix, H):
    """How a call is cut depends on all of it, so the bits may differ: each is within its bound of the
    same values, and equal calls are equal."""
    q, q64, lse, cache, qsl, seq, table, w = _inputs(cuda_device, H, q_lens, prefix, H)
    want, tol = plain.accumulate(q64, lse, cache, qsl, seq, table, BS, 64, SCALE, w)
    batch = _run(cuda_device, q, lse, cache, qsl, seq, table, w)
    _close(batch, want, tol, "batch")
    assert torch.equal(batch, _run(cuda_device, q, lse, cache, qsl, seq, table, w))
    for r in range(len(q_lens)):
        a, b = int(qsl[r]), int(qsl[r + 1])
        alone = _run(cuda_device, q[a:b], lse[a:b], cache, [0, b - a], seq[r:r + 1], table[r:r + 1], w[r:r + 1])
        _close(alone, want[r:r + 1], tol[r:r + 1], f"request {r}")


@pytest.mark.parametrize("held", [0, 1, 4, 5, 30])
@pytest.mark.parametrize("H", [8, 64])
def test_fewer_tokens_than_the_metadata_names(cuda_device, held, H):
    q, q64, lse, cache, qsl, seq, table, w = _inputs(cuda_device, held + H, [4, 60, 3], [300, 900, 20], H)
    want, tol = plain.accumulate(q64[:held], lse[:held], cache, qsl, seq, table, BS, 64, SCALE, w)
    _close(_run(cuda_device, q[:held], lse[:held], cache, qsl, seq, table, w), want, tol)
