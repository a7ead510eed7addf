"""Host-side checks of the eviction entry points (no GPU): refusals, zero work, and the plain
form by hand."""
import numpy as np
import pytest
import torch

from oracle import evict as plain
from paged_sparse_kv_gb300 import _abi, ops

INV = _abi.PSK_ERR_INVALID_ARGUMENT
OK = _abi.PSK_OK
A, B, C, D = 0x10000000, 0x20000000, 0x30000000, 0x40000000


def _select(**kw):
    a = dict(w=A, ws=100, seq=B, keep=B + 256, R=3, W=99, pos=C, ps=99, first=4, recent=8, wo=A + 2**20, wos=99, po=C + 2**20,
             pos_=100, mv=D, ms=98, nm=B + 512, so=B + 1024, err=None)
    a.update(kw)
    return _abi.status("select_cache_evictions", a["w"], a["ws"], a["seq"], a["keep"], a["R"], a["W"], a["pos"], a["ps"],
                       a["first"], a["recent"], a["wo"], a["wos"], a["po"], a["pos_"], a["mv"], a["ms"], a["nm"], a["so"],
                       a["err"], None)


@pytest.mark.parametrize("kw", [
    dict(w=None), dict(w=A + 2), dict(ws=98), dict(seq=None), dict(keep=None), dict(R=-1), dict(R=2**27 + 1), dict(W=-1),
    dict(W=2**30 + 1, ws=2**31, ps=2**31, wos=2**31, pos_=2**31, ms=2**32), dict(ps=98), dict(pos=C + 1), dict(first=-1),
    dict(recent=-1), dict(wos=98), dict(pos_=98), dict(wo=A + 1), dict(po=C + 2), dict(mv=None), dict(mv=D + 4), dict(ms=97),
    dict(ms=96), dict(nm=None), dict(so=None), dict(nm=B + 1024), dict(so=B + 256), dict(nm=B), dict(wo=A, wos=101), dict(nm=B + 1028), dict(so=B + 8), dict(so=B + 260), dict(nm=B + 4),
    dict(po=C, pos_=100), dict(err=B + 2), dict(so=B + 1)])
def test_select_rejects_bad_arguments(psk_lib, kw):
    assert _select(**kw) == INV
    assert _abi.last_error()


def test_select_no_requests_ok(psk_lib):
    assert _select(R=0, w=None, seq=None, keep=None, mv=None, nm=None, so=None) == OK


def _move(**kw):
    a = dict(c=A, np=8, ps=64 * 584, bs=64, rec=0, D=512, rope=64, ue=1, bt=B, bts=16, btw=16, base=None, R=3, mv=D, ms=64,
             M=32, nm=C, err=None)
    a.update(kw)
    return _abi.status("move_cache_rows", a["c"], a["np"], a["ps"], a["bs"], a["rec"], a["D"], a["rope"], a["ue"], a["bt"],
                       a["bts"], a["btw"], a["base"], a["R"], a["mv"], a["ms"], a["M"], a["nm"], a["err"], None)


@pytest.mark.parametrize("kw", [
    dict(c=None), dict(c=A + 8), dict(np=0), dict(ps=64 * 584 - 16), dict(bs=0), dict(rec=3), dict(rec=-1), dict(D=96),
    dict(rope=32), dict(rope=512), dict(ue=2), dict(ue=0), dict(rec=1, D=48, rope=0), dict(rec=1, D=128, rope=64), dict(bt=None),
    dict(bts=15), dict(btw=-1), dict(base=B + 2), dict(R=-1), dict(mv=None), dict(mv=D + 4), dict(ms=63), dict(ms=62),
    dict(M=-1), dict(nm=None), dict(nm=C + 2), dict(err=C + 1), dict(rec=2, D=1024, rope=0, ps=64 * 1024)])
def test_move_rejects_bad_arguments(psk_lib, kw):
    assert _move(**kw) == INV
    assert _abi.last_error()


def test_move_no_work_ok(psk_lib):
    assert _move(R=0, mv=None, nm=None, bt=None) == OK
    assert _move(M=0, ms=0, mv=None, nm=None, bt=None) == OK


def test_binding_refuses():
    w, n = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.select_cache_evictions(w, n, n)
    with pytest.raises(ValueError, match="CUDA"):
        ops.move_cache_rows(torch.zeros((2, 64), dtype=torch.uint8), n[None], torch.zeros((2, 1, 2), dtype=torch.int32), n, 1, 64)


def test_plain_form_by_hand():
    w = np.array([[5, 1, 4, 1, 0, 3, np.nan, 9]], np.float32)
    (moves, m, wo, po, err), = plain.select(w, [8], [4])
    assert (moves, m, wo, po, err) == ([(5, 1), (7, 3)], 4, [5, 3, 4, 9], [0, 5, 2, 7], False)
    # positions 0 and the newest two are protected: rows 2 (position 9), 4 (position 0) and 6 (position 8)
    p = np.array([[3, 2, 9, 4, 0, 1, 8, 5]])
    (moves, m, wo, po, _), = plain.select(w, [8], [4], p, first=1, recent=2)
    assert (moves, m, po) == ([(4, 0), (6, 1), (7, 3)], 4, [0, 8, 9, 5])
    # equals: the lower rows; none or all of them; more than there are weights for
    assert plain.select(np.zeros((1, 5), np.float32), [5], [2])[0][:2] == ([], 2)
    assert plain.select(w, [8], [0])[0][:2] == ([], 0)
    assert plain.select(w, [8], [8])[0][:2] == ([], 8)
    assert plain.select(w, [9], [4])[0][4]
    cache = np.arange(2 * 8, dtype=np.uint8).reshape(2, 8)  # pages of two records of 3 + 1 bytes
    got, errors = plain.move(cache, 2, 3, 1, np.array([[1, 0, -1]]), [[(3, 0), (4, 1)]], [2])
    assert errors == 1
    assert got.tolist() == [[0, 1, 2, 3, 4, 5, 6, 7], [3, 4, 5, 11, 12, 13, 7, 15]]
