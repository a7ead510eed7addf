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


@pytest.mark.parametrize("q_lens,prefix,H,D,window", [
    ([1], [40000], 16, 128, 20000), ([1, 2, 1], [30000, 12345, 700], 8, 128, 12000), ([300], [20000], 4, 128, 9000),
    ([5, 1], [17000, 9000], 40, 128, 16900), ([40], [9000], 16, 256, 9041), ([3], [9000], 129, 128, 8000), ([2], [100], 1, 128, 2**31 - 1)])
@pytest.mark.parametrize("decay,place", [(0.5, "in"), (1.0, "out")])
def test_long_windows(cuda_device, q_lens, prefix, H, D, window, decay, place):
    _run(cuda_device, window % 1000, q_lens, prefix, H, D, window=window, decay=decay, place=place)


@pytest.mark.parametrize("R", [60, 128, 129, 300])
def test_many_requests(cuda_device, R):
    """Tiles and rows that only fade in turn, ranges found by one warp and by all."""
    rng = np.random.default_rng(R)
    _run(cuda_device, R, rng.integers(0, 3, size=R) + (np.arange(R) == 0), rng.integers(0, 700, size=R), 16, 128, bs=16, window=40,
         decay=0.5, place="out" if R % 2 else "in")


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


def _best(call, times=4):
    """Least time of a call, in ms."""
    res = []
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        res.append(a.elapsed_time(b))
    return min(res)


def test_fading_holds_no_other_role_up(cuda_device):
    """What waits for the walk over such rows waits 2 s at most, so the walk must not do the
    fading itself: 2^28 rows took it 80 times what a plain product takes."""
    d, n = cuda_device, 1 << 28
    w = torch.ones((1, n), device=d)

    product = _best(lambda: w.mul_(0.5))
    own = _best(lambda: _no_tokens(d, w, [n], 0.5, None))
    assert own < 25 * product, (own, product)
    assert bool((w == 2.0 ** -8).all())


def test_a_window_past_the_context_is_none(cuda_device):
    """The same bits as without one, and no walk over each tile by itself (10 times the time)."""
    d, n, pages = cuda_device, 1 << 20, 1024
    g = torch.Generator("cuda").manual_seed(2)
    cache = torch.zeros((pages, 64 * 194), dtype=torch.uint8, device=d)
    cache[:, :64 * 192:2] = torch.randint(0, 0x40, (pages, 64 * 96), generator=g, device=d, dtype=torch.uint8)
    cache[:, 64 * 192:] = 127
    table = torch.randint(0, pages, (1, n // 64), generator=g, device=d, dtype=torch.int32)
    q, lse = torch.randn((1, 16, 128), generator=g, device=d).to(BF16), torch.full((1, 16), 9.0, device=d)
    args = (q, lse, cache, _i32([0, 1], d), _i32([n], d), table, 64)
    out = [torch.zeros((1, n), device=d) for _ in range(2)]
    times = [_best(lambda: ops.accumulate_attention_weights(*args, o.zero_(), window_size=w)) for o, w in zip(out, (0, n))]
    assert torch.equal(*out) and bool((out[0] > 0).all())
    assert times[1] < 3 * times[0], times
