"""apply_rotary_embedding refuses outputs whose rows share memory, and no others (no GPU: the call
that passes is stopped by its missing positions)."""
import itertools
import random

import pytest

from paged_sparse_kv_gb300 import _abi

A, B = 0x10000000, 0x20000000


def _error(tokens, heads, dim, t, h, which="q", in_place=False):
    q = (A, t, h, heads) if which == "q" else (A, dim, dim, 1)
    k = (B, t, h, heads) if which == "k" else (None, 0, 0, 0)
    shift = 0 if in_place else 2**27
    status = _abi.status("apply_rotary_embedding", *q, *k, tokens, _abi.PSK_DTYPE_BF16, dim, 0, 2, 1, 0, None, None, 2, 0,
                         q[0] + shift, q[1], q[2], None if k[0] is None else k[0] + shift, k[1], k[2], None, None)
    assert status == _abi.PSK_ERR_INVALID_ARGUMENT
    return _abi.last_error()


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens,heads,t,h", [(4, 64, 64, 64), (2, 2, 64, 64), (4, 64, 64 * 63, 64), (4, 3, 64, 65), (3, 3, 64, 130),
                                              (3, 2, 130, 260), (2, 5, 150, 70), (10**6, 128, 64, 64 * 10**6 - 1)])
def test_shared_rows_are_refused(psk_lib, tokens, heads, t, h, which, in_place):
    assert "overlap" in _error(tokens, heads, 64, t, h, which, in_place)


@pytest.mark.parametrize("tokens,heads,t,h", [(4, 64, 64 * 64, 64), (4, 64, 64, 4 * 64), (1, 9, 64, 64), (9, 1, 64, 64), (2, 2, 192, 128),
                                              (10**6, 128, 64, 64 * 10**6), (2**31 - 1, 128, 64 * 128, 64), (3, 2, 200, 100)])
def test_other_strides_pass(psk_lib, tokens, heads, t, h):
    assert "positions" in _error(tokens, heads, 64, t, h)


def test_any_strides(psk_lib):
    rng = random.Random(1)
    seen = set()
    for _ in range(3000):
        tokens, heads, dim = rng.randint(1, 6), rng.randint(1, 6), rng.choice([2, 4, 6])
        t, h = rng.randint(dim, 9 * dim), rng.randint(dim, 9 * dim)
        starts = [i * t + j * h for i, j in itertools.product(range(tokens), range(heads))]
        shared = any(abs(a - b) < dim for a, b in itertools.combinations(starts, 2))
        error = _error(tokens, heads, dim, t, h)
        assert ("overlap" in error) == shared and ("positions" in error) != shared, (tokens, heads, dim, t, h, error)
        seen.add(shared)
    assert len(seen) == 2


def test_far_strides_are_refused(psk_lib):
    """Rows whose address passes 64 bits."""
    assert "overflow" in _error(2**31 - 1, 2, 64, 2**40, 64)
    assert "overflow" in _error(2, 2**30, 64, 2**60 - 8, 2**40)


@pytest.mark.parametrize("heads,keys", [(2**31 - 1, 0), (2**31 - 2**20, 0), (2**31 - 77825, 0), (2**30, 2**30), (1, 2**31 - 2**20 - 1)])
def test_heads_past_32_bits_with_a_step(psk_lib, heads, keys):
    """A row index plus a step of all CTAs would wrap around."""
    def call(heads, keys):
        k = (B, 2 * 2**31, 2) if keys else (None, 0, 0)
        ko = (B + 2**36, *k[1:]) if keys else k
        status = _abi.status("apply_rotary_embedding", A, 2 * 2**31, 2, heads, *k, keys, 1, _abi.PSK_DTYPE_BF16, 2, 0, 2, 1, 0, None, None, 2,
                             0, A + 2**35, 2 * 2**31, 2, *ko, None, None)
        assert status == _abi.PSK_ERR_INVALID_ARGUMENT
        return _abi.last_error()
    assert "heads" in call(heads, keys)
    assert "positions" in call(2**31 - 1 - 2**20, 0) and "positions" in call(2**31 - 2**20 - 2, 1)
