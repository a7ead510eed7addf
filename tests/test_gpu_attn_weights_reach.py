"""Rows outside every new token's reach: before the windows, and of requests without tokens.
accumulate_attention_weights fades or copies them along the way."""
import numpy as np
import pytest
import torch

from paged_sparse_kv_gb300 import ops
from test_gpu_attn_weights import BF16, _i32, _run, no_wait_expires  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_lens,prefix,H,D,window", [
    ([1, 0, 2], [30000, 9000, 20011], 16, 128, 100), ([1] * 5, [129, 4000, 25000, 127, 12800], 16, 512, 128),
    ([9, 0, 0, 30], [20000, 7001, 1, 9990], 32, 128, 50), ([3], [40000], 129, 128, 1), ([0, 0, 1], [3000, 1, 0], 1, 256, 7),
    ([200, 1], [3000, 15000], 8, 256, 40)])
@pytest.mark.parametrize("decay,place", [(0.5, "in"), (1.0, "out"), (0.0, "out"), (1.0, "in")])
def test_long_contexts_short_windows(cuda_device, q_lens, prefix, H, D, window, decay, place):
    _run(cuda_device, sum(prefix), q_lens, prefix, H, D, window=window, decay=decay, place=place)


def _no_tokens(dev, w, seq, decay, out, tokens=0, H=1, window=0):
    """The call over rows without a page; `tokens` new ones of the last request."""
    R = len(seq)
    cache = torch.zeros((1, 16 * 256), dtype=torch.uint8, device=dev)
    table = torch.full((R, 1), -1, dtype=torch.int32, device=dev)
    q = torch.zeros((tokens, H, 128), dtype=BF16, device=dev)
    return ops.accumulate_attention_weights(q, torch.zeros((tokens, H), device=dev), cache, _i32([0] * R + [tokens], dev),
                                            _i32(seq, dev), table, 16, w, decay=decay, window_size=window, rope_dim=64, out=out)


@pytest.mark.parametrize("tokens,H,window", [(0, 1, 0), (1, 16, 5), (40, 64, 33)])  # the last one: pairs of CTAs
@pytest.mark.parametrize("decay,place", [(0.75, "in"), (0.75, "out"), (1.0, "out"), (0.0, "out")])
def test_millions_of_rows(cuda_device, tokens, H, window, decay, place):
    d, W = cuda_device, 3000001
    seq = [W, 0, 1, 127, 1234567, W + 5, 2500000]
    g = torch.Generator("cuda").manual_seed(1)
    big = torch.rand((len(seq), W + 3), generator=g, device=d)
    w = big[:, 1:1 + W]
    want = torch.full_like(w, -3.0) if place == "out" else w.clone()
    for r, n in enumerate(seq):
        want[r, :n] = decay * w[r, :n]
    left, right = big[:, 0].clone(), big[:, 1 + W:].clone()
    got = _no_tokens(d, w, seq, decay, torch.full_like(w, -3.0) if place == "out" else None, tokens, H, window)
    assert torch.equal(got, want)
    assert torch.equal(big[:, 0], left) and torch.equal(big[:, 1 + W:], right)


def test_fading_holds_no_other_role_up(cuda_device):
    """What waits for the walk over such rows waits 2 s at most, so the walk must not do the
    fading itself: 2^28 rows took it 80 times what a plain product takes."""
    d, n = cuda_device, 1 << 28
    w = torch.ones((1, n), device=d)

    def best(call):
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    product = best(lambda: w.mul_(0.5))
    own = best(lambda: _no_tokens(d, w, [n], 0.5, None))
    assert own < 25 * product, (own, product)
    assert bool((w == 2.0 ** -8).all())
