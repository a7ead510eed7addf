"""Host-side checks of the attention entry points (no GPU): refusals, zero work
and workspace sizes; the plain form against a hand-worked row."""
import numpy as np
import pytest

import oracle
from oracle import attention as plain
from paged_sparse_kv_gb300 import _abi

INV = _abi.PSK_ERR_INVALID_ARGUMENT
OK = _abi.PSK_OK
A, B, C = 0x10000000, 0x20000000, 0x30000000
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def _sparse(**kw):
    a = dict(q=A, qt=64 * 512, qh=512, T=4, H=64, c=B, np=8, ps=64 * 584, bs=64, x=B + 4096, xnp=4,
             xps=16 * 592, xbs=16, D=512, rope=64, idx=C, ids=640, cols=640, split=128, scale=0.1,
             sink=None, out=A + 4096, ot=64 * 512, oh=512, lse=C + 8192, ls=64, ws=C + 65536, wsb=BIG)
    a.update(kw)
    return _abi.status("sparse_mla_attention", a["q"], a["qt"], a["qh"], a["T"], a["H"], a["c"],
                       a["np"], a["ps"], a["bs"], a["x"], a["xnp"], a["xps"], a["xbs"], a["D"],
                       a["rope"], a["idx"], a["ids"], a["cols"], a["split"], a["scale"], a["sink"],
                       a["out"], a["ot"], a["oh"], a["lse"], a["ls"], a["ws"], a["wsb"], None)


COMMON = [dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 8), dict(T=-1), dict(H=0),
          dict(D=64), dict(D=1024), dict(D=96), dict(rope=16), dict(rope=512), dict(rope=-64),
          dict(qt=-8), dict(qh=12), dict(qt=4), dict(ot=256), dict(oh=504), dict(oh=516), dict(ls=63),
          dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(sink=C + 2),
          dict(lse=C + 1), dict(c=None), dict(c=B + 8), dict(np=0), dict(ps=1000), dict(bs=0),
          dict(ps=64 * 584 + 8), dict(T=2**31, ot=64 * 512)]


@pytest.mark.parametrize("kw", COMMON + [dict(idx=None), dict(idx=C + 2), dict(ids=639), dict(cols=-1),
                                         dict(split=-1), dict(split=641), dict(x=None), dict(xnp=0),
                                         dict(xps=100), dict(xbs=0), dict(x=B + 8)])
def test_sparse_rejects_bad_arguments(psk_lib, kw):
    assert _sparse(**kw) == INV
    assert _abi.last_error()


def test_sparse_zero_tokens_ok(psk_lib):
    assert _sparse(T=0, q=None, out=None, idx=None, ws=None, wsb=0) == OK
    # an extra cache is only asked for where columns name it
    assert _sparse(T=0, split=640, x=None, xnp=0, xps=0, xbs=0) == OK


def _chunk(**kw):
    a = dict(q=A, qt=64 * 512, qh=512, T=4, H=64, c=B, np=8, ps=64 * 584, bs=64, D=512, rope=64, qsl=C,
             seq=C + 64, t2r=C + 128, replay=None, R=2, bt=C + 256, bts=16, btw=16, base=None, W=128,
             valid=None, scale=0.1, sink=None, out=A + 4096, ot=64 * 512, oh=512, lse=C + 8192, ls=64,
             ws=C + 65536, wsb=BIG)
    a.update(kw)
    return _abi.status("chunk_mla_attention", a["q"], a["qt"], a["qh"], a["T"], a["H"], a["c"],
                       a["np"], a["ps"], a["bs"], a["D"], a["rope"], a["qsl"], a["seq"], a["t2r"],
                       a["replay"], a["R"], a["bt"], a["bts"], a["btw"], a["base"], a["W"],
                       a["valid"], a["scale"], a["sink"], a["out"], a["ot"], a["oh"], a["lse"],
                       a["ls"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", COMMON + [dict(qsl=None), dict(seq=None), dict(t2r=None), dict(R=0),
                                         dict(bt=None), dict(bts=15), dict(btw=-1), dict(W=-1),
                                         dict(replay=C + 2), dict(base=C + 1), dict(seq=C + 2)])
def test_chunk_rejects_bad_arguments(psk_lib, kw):
    assert _chunk(**kw) == INV
    assert _abi.last_error()


def test_chunk_zero_tokens_ok(psk_lib):
    assert _chunk(T=0, q=None, out=None, qsl=None, seq=None, t2r=None, ws=None, wsb=0) == OK


def test_workspace_sizes(psk_lib):
    s, c = psk_lib.sparse_mla_attention_workspace_bytes, psk_lib.chunk_mla_attention_workspace_bytes
    for bad in ((0, 64, 512, 640), (4, 0, 512, 640), (4, 64, 96, 640), (4, 64, 512, 0)):
        assert s(*bad) == 0
    for bad in ((0, 2, 64, 512, 16, 64, 0), (4, 0, 64, 512, 16, 64, 0), (4, 2, 64, 512, 0, 64, 0),
                (4, 2, 64, 512, 16, 64, -1)):
        assert c(*bad) == 0
    for n in (s(1, 16, 512, 640), c(2, 2, 64, 512, 2048, 64, 0)):
        assert n >= 0 and n % 16 == 0



def test_small_workspace_is_refused(psk_lib):
    n = psk_lib.sparse_mla_attention_workspace_bytes(4, 64, 512, 640)
    if n:
        assert _sparse(ws=C + 65536, wsb=n - 1) == INV
        assert _sparse(ws=None, wsb=n) == INV
        assert _sparse(ws=C + 65544, wsb=n) == INV


def test_plain_form_by_hand():
    """Two rows: k = e_0 and 2 e_1 against q = 3 e_0 + e_1, scale 1/2, sink 0."""
    D = 128
    k = np.zeros((2, D), np.float32)
    k[0, 0], k[1, 1] = 1.0, 2.0
    cache = np.zeros((1, 2 * oracle.fp8_record_bytes(D, 0) + 12), np.uint8)
    bits = (k.view(np.uint32) >> 16).astype(np.uint16)
    oracle.quantize_and_insert_k_cache(bits, np.arange(2), cache, 2, D, 0)
    q = np.zeros((1, 1, D))
    q[0, 0, 0], q[0, 0, 1] = 3.0, 1.0
    out, lse, _, _ = plain.sparse_mla_attention(q, cache, np.array([[1, -1, 0, 2]]), 2, 0, 0.5,
                                                sink=np.zeros(1))
    a, b = np.exp(1.5), np.exp(1.0)
    assert np.allclose(out[0, 0, :2], [a / (a + b + 1), 2 * b / (a + b + 1)], rtol=1e-14)
    assert np.allclose(lse[0, 0], np.log(a + b), rtol=1e-14)
