"""Tables of rotary positions against decimal arithmetic of 50 digits, within the stated bound of
m 2^-22 alone: at far positions a frequency's own error counts 2^31 times."""
import decimal
import math
from decimal import Decimal

import numpy as np
import pytest

from paged_sparse_kv_gb300 import ops

pytestmark = pytest.mark.gpu

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021")


def _frequencies(dim, theta, scaling="none", factor=1.0, original_positions=0, beta_fast=32.0, beta_slow=1.0):
    t, s = Decimal(theta), Decimal(factor)
    f = [t ** (Decimal(-2 * i) / dim) for i in range(dim // 2)]
    if scaling == "linear":
        return [x / s for x in f]
    if scaling == "yarn":
        def pair(turns):
            return dim * (original_positions / (TWO_PI * Decimal(turns))).ln() / (2 * t.ln())
        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), dim - 1)
        span = Decimal(max(hi - lo, 0)) or Decimal("0.001")
        g = [min(max((i - lo) / span, Decimal(0)), Decimal(1)) for i in range(len(f))]
        return [x * (1 - r) + x / s * r for x, r in zip(f, g)]
    return f


@pytest.mark.parametrize("dim,theta,kw", [
    (512, 1e4, {}), (512, 1e6, {}), (512, 5e5, {}), (128, 5e5, {}), (64, 1e4, {}), (64, 1.6e5, {}), (2, 1e4, {}), (34, 1.5, {}),
    (512, 1.0000001, {}), (256, 1e300, {}), (128, 1e4, dict(scaling="linear", factor=1.7)), (512, 5e5, dict(scaling="linear", factor=3.0)),
    (128, 5e5, dict(scaling="yarn", factor=40.0, original_positions=4096)),
    (512, 1e6, dict(scaling="yarn", factor=2.3, original_positions=65536)),
    (64, 1.6e5, dict(scaling="yarn", factor=16.0, original_positions=65536, attention_factor=1.2079))])
@pytest.mark.parametrize("first", [0, 1 << 20, 1 << 30, 2**31 - 24])
def test_bound(cuda_device, dim, theta, kw, first):
    n, m = 24, float(np.float32(kw.get("attention_factor", 1.0)))
    got = ops.build_rope_cos_sin_cache(n, dim, theta=theta, first_position=first, device=cuda_device, **kw).double().cpu().numpy()
    with decimal.localcontext() as c:
        c.prec = 50
        f = _frequencies(dim, theta, **{k: v for k, v in kw.items() if k != "attention_factor"})
        angle = np.array([[float((first + p) * x % TWO_PI) for x in f] for p in range(n)])
    # the reduced angle and its cosine are rounded to 2^-51 or so
    off = np.abs(got - m * np.concatenate([np.cos(angle), np.sin(angle)], 1)).max()
    assert off <= m * 2.0 ** -22, off / m * 2.0 ** 22
