"""Pools of the block-scaled cache: blocks past 2^32 bytes and elements, and blocks swapped out and in with their scales."""

import numpy as np
import pytest
import torch

from _bounded import Case

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


FAR = (1 << 18) + 5         # blocks of 16 x 8 x 128: element 2^32 is in block 2^18


def _far(c):
    """The case with every other block moved behind FAR, in pools of more than 2^32 elements, and where each went."""
    nb = c.k.shape[0]
    to = torch.arange(nb)
    to[1::2] += FAR
    shape = (FAR + nb,) + tuple(c.k.shape[1:])
    pools = []
    for x in (c.k, c.v, c.ks, c.vs):
        if x is None:
            pools.append(None)
            continue
        y = torch.empty(shape if x.dim() == 4 else (FAR + nb, x.shape[1]), dtype=x.dtype, device="cuda")
        y[to.cuda()] = x
        pools.append(y)
    tab = c.tab.cpu().long()
    inside = tab < nb
    tab = torch.where(inside, to[tab.clamp(max=nb - 1)], torch.full_like(tab, FAR + nb + 9))
    return pools, tab.int().cuda(), to.cuda()


def _same_blocks(pools, c, to):
    for y, x in zip(pools, (c.k, c.v, c.ks, c.vs)):
        if x is not None:
            a, b = y[to], x
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_blocks_past_the_32_bit_range(pa, pool):
    """The same bits as over a small pool: append, decode, kept weights, prompt attention, eviction."""
    lens = [700, 33, 150]
    c = Case(pool, lens, 16, 8, 128, 16, seed=1, codes_nan=False)
    if pool != "e4m3":
        c.k, c.v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    c.cuda()
    pools, tab, to = _far(c)
    small, big = (c.k, c.v, c.ks, c.vs), pools
    out = [torch.full_like(c.q, float("nan")) for _ in range(2)]
    w = [torch.zeros(3, 8, c.tab.shape[1] * 16, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(3)
    n = [5, 3, 130]
    if pool == "e4m3":
        key = torch.randn(sum(n), 8, 128, generator=g, device="cuda")
        q = torch.randn(sum(n), 16, 128, generator=g, device="cuda").bfloat16()
        po = [torch.full_like(q, float("nan")) for _ in range(2)]
        for i, (p, t) in enumerate(((small, c.tab), (big, tab))):
            pa.append_fp8_blocks(key, key.flip(0), _start(n).cuda(), t, c.lens, *p)
            pa.decode_fp8_blocks(out[i], c.q, *p, t, c.lens, c.scale)
            pa.prefill_fp8_blocks(po[i], q, _start(n).cuda(), *p, t, c.lens, c.scale)
        assert pa.last_error() == 0
        assert torch.equal(out[0], out[1]) and torch.equal(po[0], po[1]) and not po[0].isnan().any()
        _same_blocks(pools, c, to)
    sc = dict(k_scale=c.ks, v_scale=c.vs), dict(k_scale=big[2], v_scale=big[3])
    zero = torch.zeros_like(c.lens)
    pos = [torch.full((3, 8, c.tab.shape[1] * 16), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    new = [torch.empty_like(c.lens) for _ in range(2)]
    for i, (p, t) in enumerate(((small, c.tab), (big, tab))):
        pa.decode_weights(out[i], w[i], c.q, p[0], p[1], t, c.lens, c.scale, **sc[i])
        pa.evict(p[0], p[1], t, c.lens, zero, c.lens, w[i], pos[i], 100, new[i], w[i], pos[i], recent=10, sinks=2, **sc[i])
    assert pa.last_error() == 0
    for x in (out, w, pos, new):
        assert torch.equal(x[0], x[1])
    assert not out[0].isnan().any()
    _same_blocks(pools, c, to)


@pytest.mark.parametrize("Hkv,D", [(6, 64), (3, 128), (8, 32)])
def test_swap_out_and_in(pa, Hkv, D):
    """Codes and scales to pinned host memory and back into other blocks: the scales are fp32 pools of block size 4,
    scale_row / 4 heads and head_dim 1."""
    c = Case("e4m3", [100, 60], Hkv, Hkv, D, 16, seed=2).cuda()
    row = pa.scale_row(Hkv)
    as_pool = lambda s: s.view(s.shape[0], 4, row // 4, 1)       # noqa: E731
    host = [torch.zeros((4,) + tuple(x.shape[1:]), dtype=x.dtype).pin_memory() for x in (c.k, c.v, c.ks, c.vs)]
    was = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    src = c.tab[0, :3].tolist()
    dst = c.tab[1, 1:4].tolist()
    out = torch.tensor([[s, i + 1] for i, s in enumerate(src)], device="cuda")
    back = torch.tensor([[i + 1, d] for i, d in enumerate(dst)], device="cuda")
    pa.swap_blocks(host[0], host[1], c.k, c.v, out)
    pa.swap_blocks(as_pool(host[2]), as_pool(host[3]), as_pool(c.ks), as_pool(c.vs), out)
    torch.cuda.synchronize()
    for h, x in zip(host, was):
        assert torch.equal(h[1:].cuda(), x[src]) and not h[0].any()
    pa.swap_blocks(c.k, c.v, host[0], host[1], back)
    pa.swap_blocks(as_pool(c.ks), as_pool(c.vs), as_pool(host[2]), as_pool(host[3]), back)
    assert pa.last_error() == 0
    for x, y in zip((c.k, c.v, c.ks, c.vs), was):
        y[dst] = y[src]
        assert torch.equal(x, y)
