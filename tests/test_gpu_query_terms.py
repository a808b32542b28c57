"""Queries whose elements are far apart in size, over the block-scaled e4m3 cache: the tensor-core paths take a bf16
query as two 8-bit terms, which have to hold the small elements beside the largest."""

import numpy as np
import pytest
import torch

from _bounded import Case, check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _case(Hq, Hkv, D, bs, lens, n, small):
    """The largest element of a query meets zeros in every key; the others are `small` of it and decide."""
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=D + Hq, rows=sum(n))
    g = torch.Generator().manual_seed(7)
    held = torch.from_numpy(c.used)
    k = torch.rand(c.k.shape, generator=g) * torch.rand(c.k.shape[:2] + (1, 1), generator=g) * 448
    c.k[held] = k.to(torch.float8_e4m3fn).view(torch.uint8)[held]
    c.k[..., 0][held] = 0
    # scores up to about 20
    c.ks[:] = 2.0 ** np.round(np.log2(20 / (128 * small * D * 112 * c.scale)))
    c.q[:] = 128 * small * (1 + 7 / 128)             # the four bits that the first term leaves are 0111
    c.q[..., 1::3] = 128 * small * (1 + 55 / 128)
    c.q[..., 0] = 128.0
    return c


# exact in two terms down to 2^-13 of the largest element
@pytest.mark.parametrize("small", [2.0 ** -13, 2.0 ** -10, 2.0 ** -4])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (4, 4, 128, 8), (16, 1, 128, 32), (8, 4, 64, 16)])
def test_prefill_small_elements_beside_a_large_one(pa, Hq, Hkv, D, bs, small):
    lens, n = [200, 33, 130], [150, 33, 1]
    c = _case(Hq, Hkv, D, bs, lens, n, small)
    start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


@pytest.mark.parametrize("small", [2.0 ** -13, 2.0 ** -10, 2.0 ** -4])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (4, 4, 64, 16), (16, 4, 32, 16), (32, 2, 128, 16), (4, 2, 128, 4)])
def test_decode_small_elements_beside_a_large_one(pa, Hq, Hkv, D, bs, small):
    c = _case(Hq, Hkv, D, bs, [200, 33, 700], [1, 1, 1], small)
    ref, tol = reference(c)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)
