"""Host-side checks of accumulate_attention_weights (no GPU): refusals, zero work, the plain
form by hand."""
import numpy as np
import pytest
import torch

import oracle
from oracle import attn_weights as plain
from paged_sparse_kv_gb300 import _abi, ops

INV = _abi.PSK_ERR_INVALID_ARGUMENT
OK = _abi.PSK_OK
A, B, C, D = 0x10000000, 0x20000000, 0x30000000, 0x40000000
NAN, INF = float("nan"), float("inf")
BIG = 1 << 40


def _call(**kw):
    a = dict(q=A, qt=64 * 512, qh=512, T=4, H=64, lse=A + 2**24, ls=64, c=B, np=8, ps=64 * 584, bs=64, D=512, rope=64, qsl=C,
             seq=C + 64, replay=None, R=2, bt=C + 256, bts=16, btw=16, base=None, win=0, valid=None, scale=0.1, sink=None,
             w=D, ws=1024, W=1000, decay=1.0, out=D + 2**20, os=1000, wk=D + 2**24, wkb=BIG)
    a.update(kw)
    return _abi.status("accumulate_attention_weights", a["q"], a["qt"], a["qh"], a["T"], a["H"], a["lse"], a["ls"], a["c"],
                       a["np"], a["ps"], a["bs"], a["D"], a["rope"], a["qsl"], a["seq"], a["replay"], a["R"], a["bt"],
                       a["bts"], a["btw"], a["base"], a["win"], a["valid"], a["scale"], a["sink"], a["w"], a["ws"], a["W"],
                       a["decay"], a["out"], a["os"], a["wk"], a["wkb"], None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=A + 8), dict(qt=64 * 512 + 4), dict(qh=12), dict(qt=256), dict(qh=0), dict(qt=2**39), dict(T=-1), dict(T=2**31),
    dict(H=0), dict(H=2**21), dict(lse=None), dict(lse=A + 2), dict(ls=63), dict(c=None), dict(c=B + 8), dict(np=0), dict(ps=1000),
    dict(bs=0), dict(D=64), dict(D=1024), dict(D=192), dict(rope=32), dict(rope=512), dict(rope=-64), dict(qsl=None),
    dict(seq=None), dict(seq=C + 2), dict(replay=C + 2), dict(R=-1), dict(R=2**28), dict(bt=None), dict(bts=15), dict(btw=-1),
    dict(base=C + 1), dict(win=-1), dict(scale=0.0), dict(scale=NAN), dict(scale=INF), dict(scale=1e-40), dict(sink=C + 2),
    dict(w=None), dict(w=D + 2), dict(ws=999), dict(W=-1), dict(W=2**30 + 1, ws=2**31, os=2**31), dict(decay=-0.5), dict(decay=NAN),
    dict(decay=INF), dict(out=None), dict(out=D + 2), dict(os=999), dict(out=D, os=1000)])
def test_rejects_bad_arguments(psk_lib, kw):
    assert _call(**kw) == INV
    assert _abi.last_error()


def test_no_rows_ok(psk_lib):
    assert _call(R=0, qsl=None, seq=None, out=None, w=None) == OK
    assert _call(W=0, ws=0, os=0, out=None, w=None) == OK


def test_small_workspace_is_refused(psk_lib):
    n = psk_lib.accumulate_attention_weights_workspace_bytes()
    assert n >= 0 and n % 16 == 0
    if n:
        assert _call(wkb=n - 1) == INV
        assert _call(wk=None, wkb=n) == INV
        assert _call(wk=D + 8, wkb=n) == INV


def test_binding_refuses():
    q, n = torch.zeros((2, 1, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.accumulate_attention_weights(q, torch.zeros(2, 1), torch.zeros((1, 4096), dtype=torch.uint8), n, n[:1], n[None], 16,
                                         torch.zeros(1, 8))


def test_plain_form_by_hand():
    """Rows k = e_0, 2 e_1 and 4 e_0; two tokens whose queries are e_0 and e_1, scale 1/2, lse 0 and 1."""
    dim = 128
    k = np.zeros((3, dim), np.float32)
    k[0, 0], k[1, 1], k[2, 0] = 1.0, 2.0, 4.0
    cache = np.zeros((2, 2 * oracle.fp8_record_bytes(dim, 0) + 12), np.uint8)
    oracle.quantize_and_insert_k_cache((k.view(np.uint32) >> 16).astype(np.uint16), np.arange(3), cache, 2, dim, 0)
    q = np.zeros((2, 1, dim))
    q[0, 0, 0] = q[1, 0, 1] = 1.0
    lse = np.array([[0.0], [1.0]], np.float32)
    w = np.array([[8.0, 8.0, 8.0, 8.0]], np.float32)
    args = (q, lse, cache, [0, 2], [3], np.array([[0, 1]]), 2, 0, 0.5, w)
    out, _ = plain.accumulate(*args, decay=0.5)
    e = np.exp
    assert np.allclose(out, [[4 + e(0.5) + e(-1), 4 + e(0) + e(0), 4 + e(-1), 8]], rtol=1e-14)
    out, _ = plain.accumulate(*args, decay=0.0, sink=np.zeros(1), window=1)
    assert np.allclose(out, [[0, 1 / 2, 1 / (1 + e(1)), 8]], rtol=1e-14)
