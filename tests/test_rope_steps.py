"""pa_rope_steps against its definition in 60 decimal digits (CPU only)."""

import decimal
from decimal import Decimal

import numpy as np
import pytest

from paged_kv_cache_307_gb300 import build as B

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def pa():
    B.build()
    from paged_kv_cache_307_gb300 import _lib
    return _lib


def _turns(d, base, scaling="none", factor=1.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0):
    """f_i / 2 pi"""
    b, s = Decimal(base), Decimal(factor)
    out = []
    ln = b.ln()
    if scaling == "ntk":
        ln += s.ln() * d / (d - 2)
    edge = [d * (Decimal(original_len) / (2 * PI * Decimal(n))).ln() / (2 * ln) for n in (beta_fast, beta_slow)]
    lo, hi = max(0, edge[0].to_integral_value(decimal.ROUND_FLOOR)), min(d - 1, edge[1].to_integral_value(decimal.ROUND_CEILING))
    for i in range(d // 2):
        f = (ln * -2 * i / d).exp()
        if scaling == "linear":
            f /= s
        if scaling == "yarn":
            r = min(Decimal(1), max(Decimal(0), (i - lo) / max(hi - lo, Decimal("1e-3"))))
            f *= r / s + 1 - r
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("kw", [
    {}, dict(scaling="linear", factor=3.0), dict(scaling="ntk", factor=8.0), dict(scaling="ntk", factor=1.0),
    dict(scaling="yarn", factor=32.0), dict(scaling="yarn", factor=2.5, original_len=100.0, beta_fast=8.0, beta_slow=2.0),
    dict(scaling="yarn", factor=40.0, original_len=1e6, beta_fast=1.0, beta_slow=1.0)])
@pytest.mark.parametrize("d,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0), (512, 1e6), (32, 1.5), (48, 1.0000001), (64, 1e299)])
def test_steps_are_the_nearest(pa, kw, d, base):
    """The nearest whole number of 2^-64 turns (a remainder next to a half may go either way), so that the turn at
    every int32 position is right to 2^-33."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        steps, _ = pa.rope_steps(d, base, **kw)
        got = [int(x) for x in steps.numpy().view(np.uint64)]
        off = [abs(Decimal(g) - t * 2 ** 64) for g, t in zip(got, _turns(d, base, **kw))]
        assert max(off) <= Decimal("0.50001"), "pair %d is off by %s" % (off.index(max(off)), max(off))
