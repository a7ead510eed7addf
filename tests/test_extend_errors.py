"""What extend_block_tables counts as an error: rows that go without pages they need,
and no others.  Hand-worked, for the plain form and for the kernel."""
import numpy as np
import pytest
import torch

from oracle import batch_meta

# lengths, pages held, pool size, head; pages of 4, tables of 3 columns;
# then: pages held afterwards, head afterwards, errors
CASES = {
    "a row that does not fit, then rows that need nothing": (
        [12, 8, 4, 0], [0, 2, 1, 0], 2, 0, [0, 2, 1, 0], 0, 1),
    "a head past the pool and no demand": ([8, 4], [2, 1], 3, 4, [2, 1], 4, 0),
    "a head past the pool and one row that needs a page": ([8, 4, 4], [2, 0, 1], 3, 4, [2, 0, 1], 4, 1),
    "an empty pool and empty rows": ([0, -3, 0], [0, 0, 0], 0, 0, [0, 0, 0], 0, 0),
    "too wide for the table, past the pool": ([12, 16, 4], [0, 1, 1], 1, 0, [0, 1, 1], 0, 2),
    "after a row that does not fit, a row that would": ([12, 4], [0, 0], 2, 0, [0, 0], 0, 2),
    "the pool used up exactly, then nothing more": ([8, 4, 8], [0, 1, 2], 2, 0, [2, 1, 2], 2, 0),
}


def _table(n):
    return np.arange(3 * n).reshape(n, 3) + 100


def _want_table(table, held, before, pool, start):
    """Held columns as they were, then the pages taken, then -1."""
    want = table.copy()
    for r, (n, b) in enumerate(zip(held, before)):
        want[r, b:n] = pool[start:start + n - b]
        start += n - b
        want[r, n:] = -1
    return want


@pytest.mark.parametrize("name", CASES)
def test_plain_form(name):
    seq, before, size, head, held, head_out, errors = CASES[name]
    pool = np.arange(size) + 50
    table = _table(len(seq))
    got, counts, h, err = batch_meta.extend_block_tables(seq, pool, table, 4, counts=before, head=head)
    assert (counts.tolist(), h, err) == (held, head_out, errors)
    assert np.array_equal(got, _want_table(table, held, before, pool, head))


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_kernel(cuda_device, name):
    from paged_sparse_kv_gb300 import ops
    seq, before, size, head, held, head_out, errors = CASES[name]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=cuda_device)  # noqa: E731
    pool = np.arange(size) + 50
    table = _table(len(seq))
    err = i32([0])
    got, counts, h = ops.extend_block_tables(i32(seq), i32(pool), i32(table), 4, page_counts=i32(before),
                                             pool_head=i32([head]), err_count=err)
    assert (counts.tolist(), int(h), int(err)) == (held, head_out, errors)
    assert np.array_equal(got.cpu().numpy(), _want_table(table, held, before, pool, head))


@pytest.mark.gpu
def test_kernel_many_rows(cuda_device):
    """Several rows a CTA: the first row takes more than the pool has, the rest nothing."""
    from paged_sparse_kv_gb300 import ops
    d, R = cuda_device, 5000
    seq = torch.full((R,), 8, dtype=torch.int32, device=d)
    counts = torch.full((R,), 2, dtype=torch.int32, device=d)
    counts[0] = 0
    pool, err = torch.zeros(1, dtype=torch.int32, device=d), torch.zeros(1, dtype=torch.int32, device=d)
    table = torch.zeros((R, 3), dtype=torch.int32, device=d)
    _, held, head = ops.extend_block_tables(seq, pool, table, 4, page_counts=counts, err_count=err)
    assert int(err) == 1 and int(head) == 0 and torch.equal(held, counts)
