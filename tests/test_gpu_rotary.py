"""Rotary positions on the GPU against plain binary64 forms, within the bounds those derive
(oracle/rotary.py)."""
import numpy as np
import pytest
import torch

from oracle import rotary as plain
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}


@pytest.mark.parametrize("num,dim,first,kw", [
    (1, 2, 0, {}), (7, 6, 3, {}), (513, 64, 0, {}), (100, 64, 2**31 - 100, {}), (33, 128, 10**6, dict(theta=5e5)),
    (65, 512, 12345, {}), (40, 34, 77777, dict(scaling="linear", factor=8.0)),
    (300, 64, 10**6, dict(scaling="yarn", factor=16.0, original=65536, theta=1.6e5)),
    (50, 64, 4000, dict(scaling="yarn", factor=40.0, original=4096, beta_fast=32.0, beta_slow=1.0)),
    (50, 128, 99, dict(scaling="yarn", factor=2.5, original=3, beta_fast=1.0, beta_slow=1.0)),  # lo == hi
    (20, 64, 0, dict(attention_factor=1.2079))])
def test_table(cuda_device, num, dim, first, kw):
    want = plain.table(num, dim, kw.get("theta", 1e4), first, **{k: v for k, v in kw.items() if k != "theta"})
    own = {{"original": "original_positions"}.get(k, k): v for k, v in kw.items()}
    got = ops.build_rope_cos_sin_cache(num, dim, first_position=first, device=cuda_device, **own)
    # 2^-22 m for the value; the angle of the binary64 form is itself off by (first + num) 2^-52 or so
    tol = kw.get("attention_factor", 1.0) * 2.0 ** -22 + (first + num) * 2.0 ** -51
    assert np.abs(got.double().cpu().numpy() - want).max() <= tol


def test_table_near_axes(cuda_device):
    """Position 0 is exact; a sine near zero keeps its relative accuracy."""
    got = ops.build_rope_cos_sin_cache(2, 64, theta=1e9, device=cuda_device).double().cpu().numpy()
    assert (got[0, :32] == 1.0).all() and (got[0, 32:] == 0.0).all()
    want = plain.table(2, 64, 1e9)
    # three roundings of the angle, and those of the last two operations of the series
    assert np.abs(got[1, 32:] / want[1, 32:] - 1.0).max() <= 6 * 2.0 ** -24


def test_table_into_rows(cuda_device):
    big = torch.full((12, 80), -3.0, device=cuda_device)
    ops.build_rope_cos_sin_cache(10, 62, out=big[1:11, 5:67])
    want = plain.table(10, 62, 1e4)
    assert np.abs(big[1:11, 5:67].double().cpu().numpy() - want).max() <= 2.0 ** -22 + 10 * 2.0 ** -51
    big[1:11, 5:67] = -3.0
    assert bool((big == -3.0).all())
    assert ops.build_rope_cos_sin_cache(0, 64, device=cuda_device).shape == (0, 64)


def _make(rng, T, H, D, dtype, layout, dev):
    """A [T, H, D] tensor of a layout, its binary64 values, and the storage it is cut from."""
    x = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(dtype)
    ref = x.double().numpy()
    if layout == "thd":
        return x.to(dev), ref
    if layout == "htd":
        return x.transpose(0, 1).contiguous().to(dev).transpose(0, 1), ref
    wide = 8 if layout == "slice" else 3  # "odd": rows that start on no 16-byte boundary
    big = torch.full((T, H + 1, D + 2 * wide), 5.0, dtype=dtype)
    big[:, :H, wide:wide + D] = x
    return big.to(dev)[:, :H, wide:wide + D], ref


def _check(got, want, tol, what):
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}{i}: {g[i]}, want {want[i]} +- {tol[i]}; {bad.sum()} of {bad.size}")


def _run(dev, seed, T, H, Hk, D, offset, rope, interleaved, inverse, dtype, layout="thd", place="new", most=50):
    rng = np.random.default_rng(seed)
    cs = plain.table(most, rope, 1e4).astype(np.float32)
    pos = rng.integers(0, most, T)
    if T > 3:
        pos[[0, 2]] = -1, most  # a padding token, and one past the table
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    q, q64 = _make(rng, T, H, D, dtype, layout, dev)
    k, k64 = _make(rng, T, Hk, D, dtype, layout, dev) if Hk else (None, None)
    kw = {}
    if place == "in":
        kw = dict(q_out=q, k_out=k)
    elif place == "odd":
        kw = dict(q_out=_make(rng, T, H, D, dtype, "odd", dev)[0])
    q0, k0 = q.clone(), None if k is None else k.clone()
    qo, ko = ops.apply_rotary_embedding(torch.from_numpy(pos).to(dev), q, torch.from_numpy(cs).to(dev), k, rope_offset=offset,
                                        interleaved=interleaved, inverse=inverse, err_count=err, **kw)
    assert int(err) == (1 if T > 3 else 0)
    for got, x64, name in ((qo, q64, "q"), (ko, k64, "k")):
        if got is not None:
            want, tol = plain.rotate(x64, cs.astype(np.float64), pos, offset, interleaved, inverse, torch.finfo(dtype).eps, TINY[dtype])
            _check(got, want, tol, name)
    if place != "in":
        assert torch.equal(q, q0) and (k is None or torch.equal(k, k0))
    return q, qo


@pytest.mark.parametrize("T,H,Hk,D,offset,rope", [
    (1, 1, 0, 2, 0, 2), (1, 16, 1, 512, 448, 64), (5, 3, 2, 128, 0, 128), (4, 2, 1, 64, 5, 34), (3, 1, 1, 64, 0, 64),
    (2, 130, 1, 256, 64, 96), (9, 7, 0, 80, 16, 32), (300, 1, 1, 64, 0, 64), (6, 2, 1, 1026, 0, 1026), (700, 2, 1, 24, 8, 16)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_shapes(cuda_device, T, H, Hk, D, offset, rope, interleaved):
    for dtype in (BF16, FP16, FP32):
        _run(cuda_device, T + D, T, H, Hk, D, offset, rope, interleaved, T % 2 == 0, dtype)


@pytest.mark.parametrize("layout", ["thd", "htd", "slice", "odd"])
@pytest.mark.parametrize("place", ["new", "in", "odd"])
def test_layouts(cuda_device, layout, place):
    for dtype, interleaved in ((BF16, True), (BF16, False), (FP32, True)):
        q, _ = _run(cuda_device, 3, 5, 6, 2, 128, 64, 64, interleaved, False, dtype, layout, place)
        if layout in ("slice", "odd") and place == "in":  # nothing beside the heads is touched
            whole = q.as_strided((5, 7, q.stride(1)), q.stride(), q.storage_offset() - (8 if layout == "slice" else 3))
            whole = whole.clone()
            whole[:, :6, (8 if layout == "slice" else 3):][..., :128] = 5.0
            assert bool((whole == 5.0).all())


@pytest.mark.parametrize("seed", range(12))
def test_fuzz(cuda_device, seed):
    rng = np.random.default_rng(100 + seed)
    D = int(rng.choice([64, 128, 512, 2 * rng.integers(2, 100)]))
    rope = int(rng.choice([D, 2 * rng.integers(1, D // 2 + 1)]))
    _run(cuda_device, seed, int(rng.integers(1, 40)), int(rng.integers(1, 20)), int(rng.integers(0, 4)), D,
         int(rng.integers(0, D - rope + 1)), rope, bool(rng.integers(2)), bool(rng.integers(2)),
         (BF16, FP16, FP32)[seed % 3], str(rng.choice(["thd", "htd", "slice", "odd"])), str(rng.choice(["new", "in"])))


def test_one_head_rows(cuda_device):
    """Keys as [T, D], in place, beside queries that get an output of their own."""
    d, rng = cuda_device, np.random.default_rng(1)
    q, _ = _make(rng, 5, 4, 512, BF16, "thd", d)
    k, k64 = _make(rng, 5, 1, 512, BF16, "thd", d)
    cs = ops.build_rope_cos_sin_cache(40, 64, device=d)
    pos = torch.tensor([3, 0, 39, 7, 21], device=d)
    before = q.clone()
    q_out, k_out = ops.apply_rotary_embedding(pos, q, cs, k[:, 0], k_out=k[:, 0])
    assert k_out.shape == (5, 512) and torch.equal(q, before)
    want, tol = plain.rotate(k64, cs.double().cpu().numpy(), pos.tolist(), 448)
    _check(k_out[:, None], want, tol, "k")
    assert torch.equal(q_out[..., :448], q[..., :448]) and not torch.equal(q_out, q)


def test_special_values(cuda_device):
    """Infinities and NaN stay within their pair; dims beside and padding tokens keep their bits."""
    d = cuda_device
    cs = ops.build_rope_cos_sin_cache(8, 4, device=d)
    x = torch.ones(3, 1, 8, dtype=BF16, device=d)
    x[:, 0, 2], x[:, 0, 7] = float("inf"), float("nan")
    x[2, 0, 4] = float("nan")
    y, _ = ops.apply_rotary_embedding(torch.tensor([1, -1, 2], device=d), x, cs, rope_offset=2)
    assert torch.equal(y.view(torch.int16)[1], x.view(torch.int16)[1])
    assert torch.equal(y.view(torch.int16)[..., [0, 1, 6, 7]], x.view(torch.int16)[..., [0, 1, 6, 7]])
    assert bool(torch.isinf(y[0, 0, 2:4]).all()) and bool(torch.isfinite(y[0, 0, 4:6]).all())
    assert bool(torch.isnan(y[2, 0, 4:6]).all())


def test_inverse_is_the_adjoint(cuda_device):
    """<R x, y> = <x, R^-1 y>: the inverse is the gradient of the rotation; and R^-1 R = 1."""
    d, g = cuda_device, torch.Generator("cuda").manual_seed(3)
    x, y = (torch.randn(50, 4, 96, generator=g, device=d) for _ in range(2))
    cs = ops.build_rope_cos_sin_cache(1000, 64, device=d)
    pos = torch.randint(0, 1000, (50,), generator=g, device=d)
    for inter in (True, False):
        rx, _ = ops.apply_rotary_embedding(pos, x, cs, interleaved=inter)
        ry, _ = ops.apply_rotary_embedding(pos, y, cs, interleaved=inter, inverse=True)
        a, b = (rx.double() * y.double()), (x.double() * ry.double())
        # each term is off by at most 2^-22 of |a c| + |b s| and 2^-24 of itself
        assert abs(float(a.sum() - b.sum())) <= 2.0 ** -21 * float((rx.abs().double() + 2 * x.abs().amax()).sum() * y.abs().amax())
        back, _ = ops.apply_rotary_embedding(pos, rx, cs, interleaved=inter, inverse=True)
        # cos^2 + sin^2 of the table is off by 2 * 2^-22 sqrt(2), each rotation by 2^-22 of the pair's size
        assert float((back - x).abs().max()) <= 6 * 2.0 ** -22 * float(x.abs().max()) * 2


def test_captured_and_on_another_stream(cuda_device):
    d, g = cuda_device, torch.Generator("cuda").manual_seed(5)
    q = torch.randn(33, 8, 512, generator=g, device=d).to(BF16)
    k = torch.randn(33, 512, generator=g, device=d).to(BF16)
    cs = ops.build_rope_cos_sin_cache(100, 64, device=d)
    pos = torch.randint(0, 100, (33,), generator=g, device=d)
    want = ops.apply_rotary_embedding(pos, q, cs, k)
    torch.cuda.synchronize(d)
    s = torch.cuda.Stream(d)
    s.wait_stream(torch.cuda.current_stream(d))
    with torch.cuda.stream(s):
        other = ops.apply_rotary_embedding(pos, q, cs, k)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        table = ops.build_rope_cos_sin_cache(100, 64, device=d)
        out = ops.apply_rotary_embedding(pos, q, table, k)
    for _ in range(2):
        for o in out:
            o.fill_(-3.0)
        graph.replay()
        torch.cuda.synchronize(d)
        for w, x, y in zip(want, other, out):
            assert torch.equal(w, x) and torch.equal(w, y)


def test_refusals(cuda_device):
    d = cuda_device
    q, cs, pos = torch.zeros(4, 2, 64, dtype=BF16, device=d), torch.zeros(8, 64, device=d), torch.zeros(4, dtype=torch.int64, device=d)
    call = ops.apply_rotary_embedding
    with pytest.raises(TypeError, match="q must be"):
        call(pos, q.double(), cs)
    with pytest.raises(TypeError, match="k must be"):
        call(pos, q, cs, q.float())
    with pytest.raises(TypeError, match="positions"):
        call(pos.int(), q, cs)
    with pytest.raises(ValueError, match="4 entries"):
        call(pos[:3], q, cs)
    with pytest.raises(ValueError, match="k must be"):
        call(pos, q, cs, q[:3])
    with pytest.raises(ValueError, match="does not match"):
        call(pos, q, cs, q_out=q[:, :1])
    with pytest.raises(ValueError, match="unit inner stride"):
        call(pos, q.transpose(1, 2).contiguous().transpose(1, 2), cs)
    with pytest.raises(ValueError, match="without k"):
        call(pos, q, cs, k_out=q)
    with pytest.raises(ops.PskError):
        call(pos, q, cs, rope_offset=2)
    with pytest.raises(ops.PskError):
        call(pos, q, cs, q_out=q[:, :1].expand(4, 2, 64))  # rows of the output overlap
