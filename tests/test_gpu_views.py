"""Matrices whose rows are expanded or overlap are refused by the attention and
batch-metadata calls.  Each view lies inside an allocation that would also hold the
rows apart, so that nothing is read out of range even where a check is missing."""
import pytest
import torch

from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu

R, W = 3, 9


@pytest.mark.parametrize("which", ["expanded", "overlapping"])
def test_matrices_without_rows_of_their_own(cuda_device, which):
    d, i32 = cuda_device, torch.int32
    base = torch.zeros((R, W), dtype=i32, device=d)
    view = base[:1].expand(R, W) if which == "expanded" else base.as_strided((R, W), (W - 1, 1))
    q = torch.zeros((R, 2, 512), dtype=torch.bfloat16, device=d)
    cache = torch.zeros((2, 64 * 584), dtype=torch.uint8, device=d)
    vec, cu = torch.zeros(R, dtype=i32, device=d), torch.zeros(R + 1, dtype=i32, device=d)
    for call in (lambda: ops.sparse_mla_attention(q, cache, view, 64),
                 lambda: ops.chunk_mla_attention(q, cache, cu, vec, vec, view, 64),
                 lambda: ops.compute_slot_mappings(cu, vec, view, 64, 4),
                 lambda: ops.compute_slot_mappings(cu, vec, base, 64, 4, compressed_block_table=view)):
        with pytest.raises(ops.PskError, match="stride"):
            call()
    with pytest.raises(ValueError):
        ops.extend_block_tables(vec, vec, view, 64)


def test_single_rows_of_any_stride(cuda_device):
    """One row may carry any stride: the results of the row laid out plainly."""
    d, i32 = cuda_device, torch.int32
    row = torch.arange(W, dtype=i32, device=d)[None, :].contiguous()
    view = row.as_strided((1, W), (0, 1))
    torch.manual_seed(0)
    q = torch.randn((1, 2, 512), device=d).to(torch.bfloat16)
    cache = torch.randint(0, 100, (W, 64 * 584), dtype=torch.uint8, device=d)
    seq, cu = torch.full((1,), 70, dtype=i32, device=d), torch.tensor([0, 1], dtype=i32, device=d)
    zero = torch.zeros(1, dtype=i32, device=d)
    for call in (lambda m: ops.sparse_mla_attention(q, cache, m, 64),
                 lambda m: ops.chunk_mla_attention(q, cache, cu, seq, zero, m, 64),
                 lambda m: ops.compute_slot_mappings(cu, seq, m, 64, 4)):
        for a, b in zip(call(row), call(view)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
