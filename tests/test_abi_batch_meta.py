"""Host-side checks of the batch-metadata entry points (no GPU): refusals and
zero work, and the plain forms against hand-worked values."""
import numpy as np
import pytest

from oracle import batch_meta
from paged_sparse_kv_gb300 import _abi

INV = _abi.PSK_ERR_INVALID_ARGUMENT
OK = _abi.PSK_OK
A, B, C = 0x10000000, 0x20000000, 0x30000000


def _slots(**kw):
    a = dict(qsl=A, seq=A + 256, R=2, T=5, bt=B, bts=4, btw=4, base=None, bs=16, cbt=None, cbts=0,
             cbtw=0, cbase=None, cbs=16, ratio=4, pos=C, t2r=C + 4096, slots=C + 8192,
             comp=C + 12288)
    a.update(kw)
    return _abi.status("compute_slot_mappings", a["qsl"], a["seq"], a["R"], a["T"], a["bt"],
                       a["bts"], a["btw"], a["base"], a["bs"], a["cbt"], a["cbts"], a["cbtw"],
                       a["cbase"], a["cbs"], a["ratio"], a["pos"], a["t2r"], a["slots"],
                       a["comp"], None)


@pytest.mark.parametrize("kw", [dict(qsl=None), dict(seq=None), dict(R=0), dict(T=-1), dict(bt=None),
                                dict(bts=3), dict(btw=-1), dict(bs=0), dict(cbs=0), dict(ratio=0),
                                dict(cbt=B + 64, cbts=2, cbtw=3), dict(pos=C + 4),
                                dict(slots=C + 4), dict(comp=C + 2), dict(t2r=C + 2),
                                dict(qsl=A + 2), dict(base=A + 1), dict(cbase=A + 1),
                                dict(T=2**31)])
def test_slot_mappings_reject_bad_arguments(psk_lib, kw):
    assert _slots(**kw) == INV
    assert _abi.last_error()


def test_slot_mappings_zero_work_ok(psk_lib):
    assert _slots(T=0, qsl=None, seq=None) == OK
    assert _slots(pos=None, t2r=None, slots=None, comp=None, qsl=None) == OK


def _extend(**kw):
    a = dict(seq=A, R=3, bs=16, ratio=1, cnt=A + 256, pool=B, n=100, head=A + 512, bt=C, bts=8,
             btw=8, cnt_out=A + 1024, head_out=A + 2048, err=None)
    a.update(kw)
    return _abi.status("extend_block_tables", a["seq"], a["R"], a["bs"], a["ratio"], a["cnt"],
                       a["pool"], a["n"], a["head"], a["bt"], a["bts"], a["btw"], a["cnt_out"],
                       a["head_out"], a["err"], None)


@pytest.mark.parametrize("kw", [dict(seq=None), dict(R=-1), dict(bs=0), dict(ratio=0), dict(n=-1),
                                dict(n=2**31), dict(pool=None), dict(bt=None), dict(bts=7),
                                dict(btw=-1), dict(cnt_out=None), dict(head_out=None),
                                dict(cnt_out=A + 256), dict(cnt_out=A + 264), dict(head_out=A + 512),
                                dict(head_out=A + 260), dict(cnt_out=A + 504),
                                dict(head_out=A + 1028), dict(cnt_out=A + 8), dict(head_out=A),
                                dict(seq=A + 2), dict(err=A + 3), dict(bt=C + 2)])
def test_extend_rejects_bad_arguments(psk_lib, kw):
    assert _extend(**kw) == INV


def test_extend_zero_rows_ok(psk_lib):
    assert _extend(R=0, seq=None, cnt_out=None, head_out=None) == OK


def test_plain_slot_mappings_by_hand():
    """Two requests around an empty one, one padding token; pages of 2, ratio 3."""
    qsl, seq = [0, 2, 2, 5], [7, 9, 3]
    table = np.array([[4, 1, -1, 0], [0, 0, 0, 0], [9, 2, 5, 8]])
    pos, req, slot, comp = batch_meta.compute_slot_mappings(qsl, seq, table, 2, 6, ratio=3)
    assert pos.tolist() == [5, 6, 0, 1, 2, -1]
    assert req.tolist() == [0, 0, 2, 2, 2, -1]
    assert slot.tolist() == [-1, 0, 18, 19, 4, -1]
    assert comp.tolist() == [9, -1, -1, -1, 18, -1]  # entry 1 of page 4; entry 0 of page 9


def test_plain_extend_by_hand():
    """One row grows by two pages, one holds enough, one needs too many columns,
    one would end past the pool."""
    table = np.array([[7, -5, -5], [8, 9, -5], [-5, -5, -5], [6, -5, -5]])
    got, counts, head, errors = batch_meta.extend_block_tables(
        [11, 1, 99, 12], [30, 31, 32, 33, 34], table, 4, counts=[1, 2, 0, 1], head=2)
    assert got.tolist() == [[7, 32, 33], [8, 9, -1], [-1, -1, -1], [6, -1, -1]]
    assert (counts.tolist(), head, errors) == ([3, 2, 0, 1], 4, 2)
