"""extend_block_tables of no requests: the head comes back as a call with requests that
need nothing would give it, and only its one entry is written."""
import pytest
import torch

from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu


def _i32(a, d):
    return torch.tensor(a, dtype=torch.int32, device=d)


def _empty(d, **kw):
    return ops.extend_block_tables(_i32([], d), _i32([1, 2], d), torch.zeros((0, 3), dtype=torch.int32, device=d), 16, **kw)


@pytest.mark.parametrize("head", [None, [5], [-3], [7, 100], [-1, 4, 4]])
@pytest.mark.parametrize("entries", [None, 1, 3])
def test_head_of_no_requests(cuda_device, head, entries):
    d = cuda_device
    kw = {}
    if head is not None:
        kw["pool_head"] = _i32(head, d)
    if entries is not None:
        kw["pool_head_out"] = torch.full((entries,), -77, dtype=torch.int32, device=d)
    _, counts, got = _empty(d, **kw)
    one = ops.extend_block_tables(_i32([0], d), _i32([1, 2], d), torch.zeros((1, 3), dtype=torch.int32, device=d), 16,
                                  pool_head=kw.get("pool_head"))[2]
    assert counts.numel() == 0
    assert int(got[0]) == int(one) == max(head[0] if head else 0, 0)
    assert bool((got[1:] == -77).all())


def test_refused_calls_write_nothing(cuda_device):
    d = cuda_device
    out = _i32([9], d)
    with pytest.raises(TypeError):
        _empty(d, pool_head=torch.tensor([4], device=d), pool_head_out=out)
    with pytest.raises(ValueError):
        _empty(d, pool_head=_i32([4], d), page_counts_out=torch.zeros((2, 2), dtype=torch.int32, device=d), pool_head_out=out)
    with pytest.raises(ops.PskError):
        ops.extend_block_tables(_i32([], d), _i32([1], d), torch.zeros((0, 3), dtype=torch.int32, device=d), 0, pool_head_out=out)
    assert int(out) == 9
