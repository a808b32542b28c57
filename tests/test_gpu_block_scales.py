"""The block-scaled e4m3 cache with scales that are not powers of two, as a caller may have put there."""

import numpy as np
import pytest
import torch

import oracle
from _bounded import Case, check, reference, u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _any_scales(c, seed):
    rng = np.random.default_rng(seed)
    for s in (c.ks, c.vs):
        s.copy_(torch.from_numpy((2.0 ** -6 * (1 + rng.random(tuple(s.shape)))).astype(np.float32)))
    # (half a step of bf16 away from its values, and some that bf16 holds)
    c.vs[::3] = 2.0 ** -6 * (1 + 2.0 ** -8 - 2.0 ** -20)
    c.vs[1::5] = 2.0 ** -6 * 1.5


def _start(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)


SHAPES = [(8, 2, 128, 16), (4, 4, 128, 8), (16, 1, 128, 32), (8, 4, 64, 16), (4, 2, 128, 4)]


@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES)
def test_one_token_gives_its_value_rounded_once(pa, Hq, Hkv, D, bs):
    """The softmax of one token is 1, so the output is code * scale to the nearest bf16; decode's fp32 product and
    quotient may be off by 2^-20 of it before that rounding."""
    c = Case("e4m3", [1] * 60, Hq, Hkv, D, bs, seed=3)
    _any_scales(c, 1)
    _, V = c.f64_pools()
    ref = np.stack([np.repeat(V[int(c.tab[b, 0]), 0], Hq // Hkv, axis=0) for b in range(60)])
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, _start([1] * 60).cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    tol = (u(torch.bfloat16) + 2.0 ** -20) * np.abs(ref) + 1e-30
    check(out, ref, tol)
    out.fill_(float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    # (the tensor cores' weights, in three terms, are exact at 1)
    check(out, ref, tol + 2.0 ** -9 * np.abs(ref))


@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES)
def test_prefill_any_scale(pa, Hq, Hkv, D, bs):
    """A dequantised value is rounded to bf16 once on tensor cores: u(bf16) A on top, with A = sum p |v|."""
    lens, n = [200, 65, 300, 16], [200, 30, 5, 16]
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=5, rows=sum(n))
    _any_scales(c, 2)
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    K, V = c.f64_pools()
    tab = np.where(c.tab.numpy() < K.shape[0], c.tab.numpy(), 0)
    A = oracle.paged_prefill_varlen(c.q.double().numpy(), start.numpy(), K, np.abs(V), tab, c.lens.numpy(), c.scale)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol + u(torch.bfloat16) * A)


@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES + [(4, 4, 64, 16), (8, 4, 32, 8)])
def test_decode_any_scale(pa, Hq, Hkv, D, bs):
    c = Case("e4m3", [200, 65, 300, 16, 1000], Hq, Hkv, D, bs, seed=6)
    _any_scales(c, 3)
    ref, tol = reference(c)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


def test_prefill_nan_values_under_any_scale(pa):
    """A NaN value reaches its dim of the rows at and past its token, and no others."""
    lens, n, D, bs = [300], [300], 128, 16
    c = Case("e4m3", lens, 8, 2, D, bs, seed=5, rows=300)
    _any_scales(c, 4)
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    nan = np.zeros(c.q.shape, dtype=bool)
    for t, h, d in ((77, 1, 3), (200, 0, 127)):
        c.v[int(c.tab[0, t // bs]), t % bs, h, d] = 0xFF if t & 1 else 0x7F
        nan[t:, h * 4:(h + 1) * 4, d] = True
    c.cuda()
    out = torch.empty_like(c.q)
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    assert np.array_equal(out.isnan().cpu().numpy(), nan)
    # (u(bf16) max|v| for the values' rounding)
    check(torch.where(torch.from_numpy(nan).cuda(), torch.zeros_like(out), out), np.where(nan, 0, ref),
          tol + u(torch.bfloat16) * 448 * 2.0 ** -5)
