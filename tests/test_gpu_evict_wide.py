"""Selection for many requests of a matrix too wide for the keys of one to fit in shared memory,
with one CTA each."""
import numpy as np
import pytest

from test_gpu_evict import _select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["heavy", "ties", "any"])
@pytest.mark.parametrize("place", ["in", "out"])
def test_wide_matrix_of_many_requests(cuda_device, kind, place):
    W = 49152 + 1000
    rng = np.random.default_rng(4)
    lens = np.concatenate([rng.integers(0, 700, 58), [W, 30001]])
    keep = [int(rng.choice([max(0, n - 1), n // 8, n // 2])) for n in lens]
    _select(cuda_device, 1, W, lens.tolist(), keep, kind, first=2, recent=9, with_pos=place == "in", place=place)
