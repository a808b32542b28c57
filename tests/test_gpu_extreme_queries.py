"""Queries at the ends of bf16's range over the block-scaled e4m3 cache, with key scales that bring the scores back
to ordinary sizes."""

import numpy as np
import pytest
import torch

from _bounded import Case, check, reference
from test_gpu_bounded import _totals

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _case(Hq, Hkv, D, bs, lens, power, rows=None):
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=D + Hq, rows=rows)
    c.q *= 2.0 ** power
    c.ks *= 2.0 ** -power
    return c


SHAPES = [(8, 2, 128, 16), (16, 1, 128, 32), (4, 4, 64, 16), (8, 8, 32, 8), (4, 2, 128, 4)]


@pytest.mark.parametrize("power", [124, 115, 100, -100, -120])
@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES)
def test_decode(pa, Hq, Hkv, D, bs, power):
    c = _case(Hq, Hkv, D, bs, [200, 33, 700], power)
    assert torch.isfinite(c.q).all() and (c.ks > 0).all() and torch.isfinite(c.ks).all()
    ref, tol = reference(c)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


@pytest.mark.parametrize("power", [124, 115, 100, -100, -120])
@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES)
def test_prefill(pa, Hq, Hkv, D, bs, power):
    lens, n = [200, 33, 130], [150, 33, 1]
    c = _case(Hq, Hkv, D, bs, lens, power, rows=sum(n))
    assert torch.isfinite(c.q).all()
    start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


@pytest.mark.parametrize("power", [124, -120])
@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES + [(9, 3, 64, 16)])
def test_heads_of_one_group_far_apart(pa, Hq, Hkv, D, bs, power):
    """Every other query head at an ordinary size: its scores go to nothing, or far apart, beside the others'."""
    c = _case(Hq, Hkv, D, bs, [200, 33], power)
    c.q[:, 1::2] *= 2.0 ** (-power if power > 0 else 0)
    ref, tol = reference(c)
    start = torch.zeros(2, Hkv, c.tab.shape[1] * bs)
    wref, wtol = _totals(c, start)
    c.cuda()
    out, w = torch.full_like(c.q, float("nan")), start.cuda()
    pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs)
    assert pa.last_error() == 0
    check(out, ref, tol)
    check(w, wref, wtol)
