"""The step over a bounded cache as select_cache_evictions documents it, run as it stands there for
several steps: weights and positions are those of the rows that are there, never of rows that
have gone."""
import textwrap

import numpy as np
import pytest
import torch

from oracle import attn_weights as plain_weights
from oracle import evict as plain_evict
from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu
I32, BF16 = torch.int32, torch.bfloat16
R, H, W, KEEP, FIRST, RECENT = 3, 8, 6 * 64, 90, 4, 64


def _documented_step():
    doc = textwrap.dedent(ops.select_cache_evictions.__doc__.split("::\n", 1)[1])
    return compile(doc, "documented step", "exec")


def test_documented_step(cuda_device):
    d, rng, step = cuda_device, np.random.default_rng(3), _documented_step()
    pages = R * (W // 64)
    v = dict(ops=ops, cos_sin=ops.build_rope_cos_sin_cache(1024, 64, device=d),
             cache=torch.zeros((pages, 64 * 584), dtype=torch.uint8, device=d),
             table=torch.from_numpy(rng.permutation(pages).astype(np.int32)).to(d).view(R, -1),
             weights=torch.full((R, W), 1e3, device=d), row_positions=torch.full((R, W), 10**6, dtype=I32, device=d),
             lens=torch.zeros(R, dtype=I32, device=d), keep=torch.full((R,), KEEP, dtype=I32, device=d))
    rows = [([], []) for _ in range(R)]  # weights and positions of each request's rows
    done = [0] * R
    evicted = 0
    for new in ([120, 91, 30], [1, 1, 1], [1, 1, 70], [40, 1, 2], [1, 1, 1], [1, 25, 1], [1, 1, 1]):
        T = sum(new)
        v["q"] = torch.from_numpy(rng.standard_normal((T, H, 512)).astype(np.float32)).to(BF16).to(d)
        v["k"] = torch.from_numpy(rng.standard_normal((T, 512)).astype(np.float32)).to(BF16).to(d)
        v["positions"] = torch.from_numpy(np.concatenate([np.arange(a, a + n) for a, n in zip(done, new)])).to(d)
        v["qsl"] = torch.from_numpy(np.cumsum([0] + new).astype(np.int32)).to(d)
        # the step up to the selection, which changes the weights and the cache, is looked at in between
        seen, select = {}, ops.select_cache_evictions

        def spy(weights, *a, **kw):
            seen.update(weights=weights.cpu().numpy(), cache=v["cache"].cpu().numpy(), positions=kw["row_positions"].cpu().numpy())
            return select(weights, *a, **kw)
        ops.select_cache_evictions = spy
        try:
            exec(step, v)
        finally:
            ops.select_cache_evictions = select
        n = v["seq_lens"].tolist()
        host = np.zeros((R, W), np.float32)
        for r in range(R):
            w, p = rows[r]
            w.extend([0.0] * new[r])
            p.extend(range(done[r], done[r] + new[r]))
            done[r] += new[r]
            assert n[r] == len(w) == len(p)
            host[r, :len(w)] = w
            assert seen["positions"][r, :n[r]].tolist() == p
        want, tol = plain_weights.accumulate(v["q"].double().cpu().numpy(), v["lse"].cpu().numpy(), seen["cache"], v["qsl"].cpu().numpy(), n,
                                             v["table"].cpu().numpy(), 64, 64, np.float64(np.float32(512 ** -0.5)), host)
        got, after, now = seen["weights"], v["weights"].cpu().numpy(), v["row_positions"].cpu().numpy()
        for r in range(R):
            assert (np.abs(got[r, :n[r]] - want[r, :n[r]]) <= tol[r, :n[r]]).all()
        kept = plain_evict.select(got, n, [KEEP] * R, seen["positions"], FIRST, RECENT)
        for r, (moves, m, w, p, _) in enumerate(kept):
            assert int(v["lens"][r]) == m
            assert after[r, :m].tolist() == [float(x) for x in w] and now[r, :m].tolist() == p
            rows[r] = ([float(x) for x in w], list(p))
            evicted += n[r] - m
    assert evicted > 100
