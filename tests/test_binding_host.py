"""What the binding hands to the C ABI, recorded on the CPU: nothing is launched.

The addresses are those of CPU tensors; a recorder stands in for the call."""
import pytest
import torch

from paged_sparse_kv_gb300 import _abi, ops

I32 = torch.int32


@pytest.fixture
def recorded(monkeypatch):
    """Calls as (name, arguments); CPU tensors pass as device -1."""
    calls = []
    monkeypatch.setattr(ops, "_index", lambda t: t.get_device())
    monkeypatch.setattr(ops, "_on", lambda index, fn, *args: 0)
    monkeypatch.setattr(ops._abi, "lib", lambda: _NoLibrary)
    monkeypatch.setattr(ops, "_call", lambda dev, name, *args: calls.append((name, args)))
    return calls


class _NoLibrary:
    sparse_mla_attention_workspace_bytes = chunk_mla_attention_workspace_bytes = None


# Where each call has the row strides of its matrices, by position in its C argument list.
SPARSE_IDX_STRIDE, CHUNK_BT_STRIDE, SLOTS_BT_STRIDE, SLOTS_COMP_BT_STRIDE = 16, 17, 5, 10


def _views(rows, width):
    """Matrices of `rows` equal rows that are one row in memory, and of rows that overlap."""
    base = torch.zeros((rows, width), dtype=I32)
    return [base[:1].expand(rows, width), base.as_strided((rows, width), (width - 1, 1))]


def _q(T):
    return torch.zeros((T, 2, 512), dtype=torch.bfloat16)


CACHE = torch.zeros((2, 64 * 584), dtype=torch.uint8)


@pytest.mark.parametrize("which", [0, 1])
def test_strides_of_views_are_passed_as_they_are(recorded, which):
    """A stride below the width reaches the C ABI, which refuses it: rounded up to the
    width, the kernel would read rows that do not exist."""
    R, W = 3, 9
    want = (0, W - 1)[which]
    view = _views(R, W)[which]
    vec, cu = torch.zeros(R, dtype=I32), torch.zeros(R + 1, dtype=I32)
    ops.sparse_mla_attention(_q(R), CACHE, view, 64)
    ops.chunk_mla_attention(_q(R), CACHE, cu, vec, vec, view, 64)
    ops.compute_slot_mappings(cu, vec, view, 64, 4, compressed_block_table=view)
    (_, sparse), (_, chunk), (_, slots) = recorded
    assert sparse[SPARSE_IDX_STRIDE:SPARSE_IDX_STRIDE + 2] == (want, W)
    assert chunk[CHUNK_BT_STRIDE:CHUNK_BT_STRIDE + 2] == (want, W)
    assert slots[SLOTS_BT_STRIDE:SLOTS_BT_STRIDE + 2] == (want, W)
    assert slots[SLOTS_COMP_BT_STRIDE:SLOTS_COMP_BT_STRIDE + 2] == (want, W)


@pytest.mark.parametrize("rows,width,stride", [(1, 9, 9), (3, 0, 0), (3, 9, 12)])
def test_strides_of_ordinary_matrices(recorded, rows, width, stride):
    """One row of any stride, no columns, and rows apart from each other stay accepted."""
    view = torch.zeros((rows, 12), dtype=I32)[:, :width]
    if rows == 1:
        view = view.as_strided((1, width), (0, 1))
    vec, cu = torch.zeros(rows, dtype=I32), torch.zeros(rows + 1, dtype=I32)
    ops.sparse_mla_attention(_q(rows), CACHE, view, 64)
    ops.chunk_mla_attention(_q(rows), CACHE, cu, vec, vec, view, 64)
    ops.compute_slot_mappings(cu, vec, view, 64, 4)
    (_, sparse), (_, chunk), (_, slots) = recorded
    assert sparse[SPARSE_IDX_STRIDE:SPARSE_IDX_STRIDE + 2] == (stride, width)
    assert chunk[CHUNK_BT_STRIDE:CHUNK_BT_STRIDE + 2] == (stride, width)
    assert slots[SLOTS_BT_STRIDE:SLOTS_BT_STRIDE + 2] == (stride, width)


def test_recorded_positions_match_the_signatures():
    """The arguments the tests above pick are 64-bit strides followed by 32-bit widths."""
    for name, at in (("sparse_mla_attention", SPARSE_IDX_STRIDE), ("chunk_mla_attention", CHUNK_BT_STRIDE),
                     ("compute_slot_mappings", SLOTS_BT_STRIDE), ("compute_slot_mappings", SLOTS_COMP_BT_STRIDE)):
        args = _abi.SIGNATURES[name][1]
        assert args[at - 1] is _abi._P and args[at] is _abi._I64 and args[at + 1] is _abi._I32, name
