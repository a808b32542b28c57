"""The block-scaled cache, kept weights and eviction at sizes where the kernels' rings, slots, chunks and loops come
round again: contexts of many key tiles, many partitions, wide tables, many destination blocks."""

import numpy as np
import pytest
import torch

from _bounded import Case, check, reference
from test_gpu_bounded import _evict_both, _evict_inputs, _totals

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


# ------------------------------------------------------------------ prompt attention over many key tiles

@pytest.mark.parametrize("Hq,Hkv,bs", [(2, 2, 16), (8, 2, 16), (16, 1, 8), (4, 1, 32), (6, 2, 16)])
@pytest.mark.parametrize("lens,n", [([385, 513, 1100], [385, 300, 520]), ([2000], [130]), ([2000, 900], [1, 600]),
                                    ([1537, 640, 641, 768, 769], [17, 1, 65, 129, 257])])
def test_prefill_many_key_tiles(pa, Hq, Hkv, bs, lens, n):
    c = Case("e4m3", lens, Hq, Hkv, 128, bs, seed=Hq + len(lens), rows=sum(n))
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


def test_prefill_scales_that_change_from_tile_to_tile(pa):
    """Each block's scales are its own: a slot read a turn early or late shows."""
    lens, n = [1700], [300]
    c = Case("e4m3", lens, 8, 2, 128, 16, seed=1, rows=300)
    rng = np.random.default_rng(5)
    c.ks[:] = torch.exp2(torch.from_numpy(rng.integers(-12, -4, tuple(c.ks.shape)).astype(np.float32)))
    c.vs[:] = torch.exp2(torch.from_numpy(rng.integers(-12, 3, tuple(c.vs.shape)).astype(np.float32)))
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


# ------------------------------------------------------------------ kept weights over chunks and partitions

def _weights(pa, c, partition, slots=None):
    ref, tol = reference(c)
    g = torch.Generator().manual_seed(1)
    start = torch.rand(len(c.lens), c.Hkv, slots or c.tab.shape[1] * c.bs, generator=g)
    wref, wtol = _totals(c, start)
    c.cuda()
    out, w = torch.full_like(c.q, float("nan")), start.cuda()
    pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs,
                      partition_size=partition)
    assert pa.last_error() == 0
    check(out, ref, tol)
    check(w, wref, wtol)
    for b, L in enumerate(c.lens.tolist()):
        assert torch.equal(w[b, :, L:].cpu(), start[b, :, L:])


@pytest.mark.parametrize("pool,Hq,Hkv,D,bs", [("f32", 6, 2, 64, 16), ("bf16", 8, 2, 128, 16), ("bf16", 3, 1, 128, 32),
                                              ("e4m3", 8, 2, 128, 16), ("e4m3", 4, 4, 64, 8), ("e4m3", 5, 1, 64, 16),
                                              ("e4m3", 16, 1, 128, 16)])
@pytest.mark.parametrize("partition", [0, 64, -1])
def test_weights_over_several_chunks(pa, pool, Hq, Hkv, D, bs, partition):
    """1024 tokens a chunk; at 64 tokens a partition more partitions than a warp has lanes."""
    _weights(pa, Case(pool, [1025, 2049, 5000, 1024, 3], Hq, Hkv, D, bs, seed=bs + D), partition)


@pytest.mark.parametrize("pool", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("spare,lens", [(320, [3000, 1025]), (1900, [9000, 20])])
def test_weights_wide_tables_take_several_chunks_a_cta(pa, pool, spare, lens):
    """64 sequences x 8 heads: tables of 5 and of 20 thousand tokens and more make several chunks a CTA's."""
    rng = np.random.default_rng(3)
    lens = lens + rng.integers(0, 90, 62).tolist()
    c = Case(pool, lens, 16, 8, 64, 16, seed=9, spare_cols=spare)
    assert 64 * 8 * -(-c.tab.shape[1] * 16 // 1024) >= 2 * 8 * 152
    _weights(pa, c, 0)


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (3, 3, 64, 8), (8, 4, 32, 16), (4, 2, 128, 4)])
@pytest.mark.parametrize("partition", [32, 192, 4096])
def test_decode_many_partitions(pa, Hq, Hkv, D, bs, partition):
    c = Case("e4m3", [5000, 1100, 700, 2], Hq, Hkv, D, bs, seed=4)
    ref, tol = reference(c)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale, partition_size=partition)
    assert pa.last_error() == 0
    check(out, ref, tol)


# ------------------------------------------------------------------ eviction into many blocks

@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("budget,extra", [(640, 100), (1100, 40), (150, 90)])
def test_evict_many_rows_and_destination_blocks(pa, pool, budget, extra):
    """320 (sequence, head) rows, for which a CTA of the second kernel takes 32 destination blocks."""
    rng = np.random.default_rng(budget)
    lens = (budget + rng.integers(-20, extra, 40)).tolist()
    args = _evict_inputs(pool, lens, 8, 32, 16, budget, seed=2, kept=range(0, 40, 3))
    assert _evict_both(pa, *args, budget, 30, 4, False) == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_evict_few_rows_and_many_destination_blocks(pa, pool):
    args = _evict_inputs(pool, [3000, 2500, 1900], 2, 64, 16, 1700, seed=4, kept=(1,))
    assert _evict_both(pa, *args, 1700, 100, 4, True) == 0
