"""Slot maps on both sides of the rule that gives a thread two tokens, and with outputs
left out at the C ABI."""
import numpy as np
import pytest
import torch

from oracle import batch_meta
from paged_sparse_kv_gb300 import _abi, ops

pytestmark = pytest.mark.gpu

BS, RATIO = 64, 4
DTYPES = (torch.int64, torch.int32, torch.int64, torch.int64)


def _case(d, T, R, seed):
    """Inputs of T tokens, the last two of them padding, and the plain form's outputs."""
    rng = np.random.default_rng(seed)
    q = np.bincount(rng.integers(0, R, size=T - 2), minlength=R)
    seq = (q + rng.integers(0, 300, size=R)).astype(np.int32)
    qsl = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    table = rng.integers(-1, 1000, size=(R, int(seq.max()) // BS + 1)).astype(np.int32)
    want = batch_meta.compute_slot_mappings(qsl, seq, table, BS, T, ratio=RATIO)
    return [torch.from_numpy(a).to(d) for a in (qsl, seq, table)], want


@pytest.mark.parametrize("off", [-1, 0, 1])
def test_both_sides_of_two_tokens_a_thread(cuda_device, off):
    """Two from 6 x 256 tokens per SM on."""
    T = torch.cuda.get_device_properties(cuda_device).multi_processor_count * 6 * 256 + off
    (qsl, seq, table), want = _case(cuda_device, T, 3, T)
    got = ops.compute_slot_mappings(qsl, seq, table, BS, T, compress_ratio=RATIO)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("T", [3001, 250001])
@pytest.mark.parametrize("given", range(1, 16))
def test_outputs_left_out(cuda_device, T, given):
    """Every choice of the four outputs, with the entries behind them left as they were."""
    d = cuda_device
    (qsl, seq, table), want = _case(d, T, 3, 7)
    outs = [torch.full((T + 4,), -77, dtype=t, device=d) if given >> i & 1 else None for i, t in enumerate(DTYPES)]
    _abi.call("compute_slot_mappings", qsl.data_ptr(), seq.data_ptr(), 3, T, table.data_ptr(), table.stride(0),
              table.shape[1], None, BS, None, 0, 0, None, BS, RATIO, *(None if o is None else o.data_ptr() for o in outs),
              torch.cuda.current_stream(d).cuda_stream)
    for o, w in zip(outs, want):
        if o is not None:
            assert np.array_equal(o[:T].cpu().numpy(), w) and bool((o[T:] == -77).all())
