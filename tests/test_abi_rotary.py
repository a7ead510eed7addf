"""Host-side checks of the rotary entry points (no GPU): refusals, zero work, and the plain
form against hand-worked values."""
import numpy as np
import pytest
import torch

from oracle import rotary as plain
from paged_sparse_kv_gb300 import _abi, ops

INV = _abi.PSK_ERR_INVALID_ARGUMENT
OK = _abi.PSK_OK
A, B, C = 0x10000000, 0x20000000, 0x30000000
NAN, INF = float("nan"), float("inf")


def _table(**kw):
    a = dict(out=A, cs=64, first=0, n=16, rope=64, theta=1e4, scaling=0, factor=1.0, orig=0, fast=32.0, slow=1.0, m=1.0)
    a.update(kw)
    return _abi.status("build_rope_cos_sin_cache", a["out"], a["cs"], a["first"], a["n"], a["rope"], a["theta"],
                       a["scaling"], a["factor"], a["orig"], a["fast"], a["slow"], a["m"], None)


@pytest.mark.parametrize("kw", [
    dict(out=None), dict(out=A + 2), dict(cs=63), dict(first=-1), dict(n=-1), dict(first=2**31), dict(n=2**31 + 1),
    dict(rope=0), dict(rope=63), dict(rope=514, cs=514), dict(rope=-2), dict(theta=1.0), dict(theta=NAN), dict(theta=INF),
    dict(scaling=3), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=NAN),
    dict(scaling=2, factor=4.0, orig=0), dict(scaling=2, factor=INF, orig=4096),
    dict(scaling=2, factor=4.0, orig=4096, slow=0.0), dict(scaling=2, factor=4.0, orig=4096, fast=0.5),
    dict(m=0.0), dict(m=-1.0), dict(m=NAN), dict(m=1e60), dict(cs=2**60)])
def test_table_rejects_bad_arguments(psk_lib, kw):
    assert _table(**kw) == INV
    assert _abi.last_error()


def test_table_no_positions_ok(psk_lib):
    assert _table(n=0, out=None) == OK


def _apply(**kw):
    a = dict(q=A, qt=64 * 512, qh=512, H=64, k=B, kt=512, kh=512, Hk=1, T=4, dt=0, D=512, off=448, rope=64, inter=1,
             inv=0, pos=C, cs=C + 4096, css=64, most=100, qo=A + 2**26, qot=64 * 512, qoh=512, ko=B + 2**26, kot=512,
             koh=512, err=None)
    a.update(kw)
    return _abi.status("apply_rotary_embedding", a["q"], a["qt"], a["qh"], a["H"], a["k"], a["kt"], a["kh"], a["Hk"],
                       a["T"], a["dt"], a["D"], a["off"], a["rope"], a["inter"], a["inv"], a["pos"], a["cs"], a["css"],
                       a["most"], a["qo"], a["qot"], a["qoh"], a["ko"], a["kot"], a["koh"], a["err"], None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(qo=None), dict(q=A + 1), dict(qo=A + 1), dict(k=B + 1), dict(ko=None), dict(H=0), dict(Hk=0), dict(T=-1),
    dict(T=2**31), dict(dt=3), dict(dt=-1), dict(dt=2, q=A + 2), dict(D=1), dict(D=2**17), dict(rope=0), dict(rope=63),
    dict(rope=-2), dict(off=-1), dict(off=449), dict(inter=2), dict(inv=-1), dict(css=63), dict(most=-1), dict(pos=None),
    dict(pos=C + 4), dict(cs=None), dict(cs=C + 2), dict(qt=-1), dict(qoh=-512), dict(qot=511), dict(qoh=511), dict(kot=8),
    dict(qo=A, qot=65 * 512), dict(qo=A, qoh=520), dict(ko=B, kot=520), dict(err=C + 2), dict(kt=2**62),
    dict(H=2**31 - 1, Hk=1)])
def test_apply_rejects_bad_arguments(psk_lib, kw):
    assert _apply(**kw) == INV
    assert _abi.last_error()


def test_apply_zero_tokens_ok(psk_lib):
    assert _apply(T=0, q=None, qo=None, pos=None, cs=None) == OK


def test_binding_refuses():
    x, p, cs = torch.zeros(3, 2, 8), torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.apply_rotary_embedding(p, x, cs)
    with pytest.raises(ValueError, match="scaling"):
        ops.build_rope_cos_sin_cache(4, 8, scaling="ntk")
    with pytest.raises(ValueError, match="CUDA"):
        ops.build_rope_cos_sin_cache(4, 8, device="cpu")
    with pytest.raises(ValueError, match=">= 0"):
        ops.build_rope_cos_sin_cache(-1, 8)


def test_plain_form_by_hand():
    # quarter turns: (a, b) -> (-b, a), and back
    cs = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    got, _ = plain.rotate(x, cs, [1], 1)
    assert got.tolist() == [[[1, -3, 2, -5, 4, 6]]]
    got, _ = plain.rotate(x, cs, [1], 1, interleaved=False)
    assert got.tolist() == [[[1, -4, -5, 2, 3, 6]]]
    assert plain.rotate(got, cs, [1], 1, interleaved=False, inverse=True)[0].tolist() == x.tolist()
    assert plain.rotate(x, cs, [-1], 1)[0].tolist() == plain.rotate(x, cs, [2], 1)[0].tolist() == x.tolist()
    # frequencies 1 and 1/100; by parts with a ramp from pair 0 to 1: the first as it is, the second stretched
    assert plain.frequencies(4, 1e4) == [1.0, 0.01]
    assert np.allclose(plain.frequencies(4, 1e4, "linear", 4.0), [0.25, 0.0025], rtol=1e-15)
    f = plain.frequencies(4, 1e4, "yarn", 4.0, 200.0, beta_fast=32.0, beta_slow=1.0)
    # d(32) = 4 ln(200 / 64 pi) / (2 ln 1e4) < 0 -> 0; d(1) = 4 ln(31.8) / 18.4 = 0.75 -> 1
    assert np.allclose(f, [1.0, 0.0025], rtol=1e-15)
