"""Calls of the block-scaled cache that are allowed and rare: one row in all, large query groups, queries that are not
finite, empty sequences in a padded batch, captured and replayed calls, calls on a stream of their own."""

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


def _start(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)


def _cache(c):
    return c.k, c.v, c.ks, c.vs


@pytest.mark.parametrize("lens,n", [([1], [1]), ([300], [1]), ([0, 77, 0], [0, 1, 0]), ([5, 0, 130, 0, 40], [5, 0, 3, 0, 0])])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(4, 4, 128, 16), (65, 1, 128, 16), (100, 1, 128, 8), (256, 2, 128, 16),
                                         (129, 1, 128, 16), (6, 2, 64, 4)])
def test_prefill_few_rows_and_large_groups(pa, Hq, Hkv, D, bs, lens, n):
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=Hq, rows=sum(n))
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), *_cache(c), c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (4, 4, 64, 16), (8, 4, 32, 16), (4, 2, 128, 4), (40, 2, 128, 16)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_not_finite_keeps_to_its_row_and_head(pa, Hq, Hkv, D, bs, value):
    lens, n = [150, 40], [20, 3]
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=6, rows=23)
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    c.q[5, 1, 7] = value
    c.cuda()
    out = torch.empty_like(c.q)
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), *_cache(c), c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    nan = np.zeros(c.q.shape, dtype=bool)
    nan[5, 1] = True
    assert np.array_equal(out.isnan().cpu().numpy(), nan)
    check(torch.where(torch.from_numpy(nan).cuda(), torch.zeros_like(out), out), np.where(nan, 0, ref), tol)
    # the same rows' last tokens as decode
    d = Case("e4m3", lens, Hq, Hkv, D, bs, seed=6)
    ref, tol = reference(d)
    d.q[1, Hq - 1, 0] = value
    d.cuda()
    out = torch.empty_like(d.q)
    pa.decode_fp8_blocks(out, d.q, *_cache(d), d.tab, d.lens, d.scale)
    assert pa.last_error() == 0
    nan = np.zeros(d.q.shape, dtype=bool)
    nan[1, Hq - 1] = True
    assert np.array_equal(out.isnan().cpu().numpy(), nan)
    check(torch.where(torch.from_numpy(nan).cuda(), torch.zeros_like(out), out), np.where(nan, 0, ref), tol)


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (4, 2, 64, 16)])
def test_captured_append_and_prompt_attention(pa, Hq, Hkv, D, bs):
    """Chunks of two prompts, appended and attended to, by one graph replayed with other rows and lengths: the bits
    of the eager calls."""
    def run(graph):
        c = Case("e4m3", [400, 300], Hq, Hkv, D, bs, seed=1).cuda()
        start = _start([40, 24]).cuda()
        key, val = (torch.zeros(64, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.zeros(64, Hq, D, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        lens = torch.tensor([40, 24], dtype=torch.int32, device="cuda")

        def chunk():
            pa.append_fp8_blocks(key, val, start, c.tab, lens, *_cache(c))
            pa.prefill_fp8_blocks(out, q, start, *_cache(c), c.tab, lens, c.scale)
        if graph:
            g = torch.cuda.CUDAGraph()
            chunk()                                  # (what is set up once is set up)
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                chunk()
        gen = torch.Generator(device="cuda").manual_seed(4)
        outs = []
        lens.zero_()
        for _ in range(9):
            lens += torch.tensor([40, 24], dtype=torch.int32, device="cuda")
            for x in (key, val, q):
                x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            g.replay() if graph else chunk()
            outs.append(out.clone())
        torch.cuda.synchronize()
        assert pa.last_error() == 0
        held = [x[c.tab[b, :n // bs].long()] for b, n in ((0, 360), (1, 216)) for x in _cache(c)]
        return outs + [x[..., :Hkv] if x.dim() == 2 else x for x in held]
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_every_call_on_a_stream_of_its_own(pa):
    """A step's calls on another stream than the current one, each making its own workspace, while the current stream
    fills and frees memory."""
    def run(side):
        c = Case("e4m3", [200, 61, 130], 8, 2, 128, 16, seed=3, codes_nan=False).cuda()
        w = torch.zeros(3, 2, c.tab.shape[1] * 16, device="cuda")
        pos = torch.full(w.shape, -1, dtype=torch.int32, device="cuda")
        zero, out = torch.zeros_like(c.lens), torch.zeros_like(c.q)
        new, o2 = torch.empty_like(c.lens), torch.zeros_like(c.q)
        key = torch.randn(3, 2, 128, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
        st = _start([1, 1, 1]).cuda()
        torch.cuda.synchronize()
        at = dict(stream=side)
        for _ in range(3):
            if side is not None:
                for k in range(10):
                    torch.full((1 << (8 + k),), 0x7F, dtype=torch.uint8, device="cuda")
            pa.append_fp8_blocks(key, key, st, c.tab, c.lens, *_cache(c), **at)
            pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs, **at)
        pa.evict(c.k, c.v, c.tab, c.lens, zero, c.lens, w, pos, 50, new, w, pos, recent=5, k_scale=c.ks, v_scale=c.vs,
                 **at)
        pa.decode_fp8_blocks(o2, c.q, *_cache(c), c.tab, new, c.scale, **at)
        torch.cuda.synchronize()
        assert pa.last_error() == 0
        return [out, o2, w, pos, new] + [x.view(torch.uint8) for x in _cache(c)]
    for a, b in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(a, b)
