"""Plain binary64 forms of the rotary-position steps (test infrastructure): one pair
at a time from the definition, with bounds on what binary32 arithmetic and one
rounding to the tensor's type may be off by."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rope_dim, theta, scaling="none", factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    f = [theta ** (-2.0 * i / rope_dim) for i in range(rope_dim // 2)]
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling == "yarn":
        def pair(turns):
            return rope_dim * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), rope_dim - 1)
        span = max(hi - lo, 0.001)
        g = [min(max((i - lo) / span, 0.0), 1.0) for i in range(len(f))]
        return [x * (1 - r) + x / factor * r for x, r in zip(f, g)]
    return f


def table(num, rope_dim, theta, first=0, attention_factor=1.0, **kw):
    """[num, rope_dim] in binary64."""
    a = np.arange(first, first + num, dtype=np.float64)[:, None] * np.array(frequencies(rope_dim, theta, **kw))
    return np.concatenate([np.cos(a), np.sin(a)], 1) * attention_factor


def rotate(x, cos_sin, positions, offset, interleaved=True, inverse=False, eps=2.0 ** -7, tiny=0.0):
    """x [T, H, D] binary64 of type values; returns (out, bound).

    Bound: two products and a sum in binary32, each off by 2^-24 of the products' sizes,
    then a rounding to the type, eps / 2 of the result or half the smallest step."""
    T, H, D = x.shape
    n = cos_sin.shape[1] // 2
    out, tol = x.copy(), np.zeros_like(x)
    for t in range(T):
        p = int(positions[t])
        if not 0 <= p < cos_sin.shape[0]:
            continue
        for i in range(n):
            c, s = float(cos_sin[p, i]), float(cos_sin[p, n + i]) * (-1 if inverse else 1)
            ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + n + i)
            a, b = x[t, :, ia], x[t, :, ib]
            for at, y, size in ((ia, a * c - b * s, abs(a * c) + abs(b * s)), (ib, b * c + a * s, abs(b * c) + abs(a * s))):
                out[t, :, at] = y
                tol[t, :, at] = np.abs(y) * (eps / 2) * 1.01 + size * 2.0 ** -22 + tiny
    return out, tol
