"""The block-scaled e4m3 cache through the C ABI against the oracle: append bit for bit, decode and causal
attention within tolerances derived in _bounded.py."""

import numpy as np
import pytest
import torch

import oracle
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


# ------------------------------------------------------------------ append

def _append_case(lens, new, Hkv, D, bs, dt, seed=0):
    c = Case("e4m3", lens, Hkv, Hkv, D, bs, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    T = int(sum(new))
    size = torch.exp2(torch.randint(-9, 9, (T, Hkv, 1), generator=g).float())
    key = (torch.randn(T, Hkv, D, generator=g) * size).to(dt)
    val = (torch.randn(T, Hkv, D, generator=g) * size.flip(0)).to(dt)
    return c, key, val, _start(new)


def _append_both(pa, c, key, val, start):
    ref = oracle.append_fp8_blocks(key.double().numpy(), val.double().numpy(), start.numpy(), c.tab.numpy(),
                                   c.lens.numpy(), c.k.numpy(), c.v.numpy(), c.ks.numpy(), c.vs.numpy())
    got = [x.cuda() for x in (c.k, c.v, c.ks, c.vs)]
    pa.append_fp8_blocks(key.cuda(), val.cuda(), start.cuda(), c.tab.cuda(), c.lens.cuda(), *got)
    return got, ref


@pytest.mark.parametrize("Hkv,D,bs", [(2, 128, 16), (8, 128, 16), (3, 64, 8), (1, 32, 4), (5, 128, 32), (40, 64, 16)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_append_bit_exact(pa, Hkv, D, bs, dt):
    lens = [1, bs, bs + 1, 3 * bs - 1, 5 * bs, 70, 33]
    new = [1, 1, 1, 2 * bs, 5 * bs, 0, 32]
    got, ref = _append_both(pa, *_append_case(lens, new, Hkv, D, bs, dt))
    assert pa.last_error() == 0
    for g, r in zip(got, ref):
        assert np.array_equal(g.cpu().numpy(), r)


def test_append_steps_equal_one_call(pa):
    """Token by token, the codes are those of one call wherever the values stay normal under the final scale."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randint(0, 2, (37, 4, 128), generator=g) * 2 - 1) * torch.exp2(torch.rand(37, 4, 128, generator=g) * 6)
    x = x.to(torch.bfloat16).cuda()
    tab = torch.randperm(6, generator=g).int().view(1, 6)[:, :3].contiguous().cuda()
    pools = []
    for splits in ([37], [1] * 37, [5, 16, 1, 15]):
        k = [torch.zeros(6, 16, 4, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.zeros(6, 4, device="cuda") for _ in range(2)]
        done = 0
        for n in splits:
            part = x[done:done + n].contiguous()
            done += n
            pa.append_fp8_blocks(part, part, _start([n]).cuda(), tab, torch.tensor([done], dtype=torch.int32).cuda(),
                                 *k, *s)
        pools.append(k + s)
    assert pa.last_error() == 0
    for p in pools[1:]:
        assert all(torch.equal(a, b) for a, b in zip(p, pools[0]))


def test_append_zeros_extremes_and_not_finite(pa):
    c, key, val, start = _append_case([16, 17, 20, 9], [16, 17, 3, 9], 2, 64, 16, torch.float32)
    key[:16] = 0.0                                   # a block of nothing but zeros
    key[16:33] = 3e38                                # the largest magnitudes
    val[16:33] *= 1e-38                              # magnitudes below the smallest scale's range
    key[33, 0, 5], key[34, 1, 0] = float("inf"), float("-inf")
    val[35, 0, 1] = float("nan")
    got, ref = _append_both(pa, c, key, val, start)
    assert pa.last_error() == 0
    for g, r in zip(got, ref):
        g = g.cpu().numpy()
        if g.dtype == np.uint8:
            g, r = (np.where((x & 0x7F) == 0x7F, 0x7F, x) for x in (g, r))    # a NaN code of either sign
        assert np.array_equal(g, r)
    assert float(got[2][c.tab[0, 0].long(), 0]) == 0.0


def test_append_bad_arguments_on_the_device_write_nothing(pa):
    c, key, val, start = _append_case([20, 20, 20, 20], [4, 4, 4, 4], 2, 64, 16, torch.bfloat16)
    for change, bit in ((dict(lens=[20, -1, 20, 20]), pa.DEV_BAD_LEN), (dict(lens=[20, 10 ** 6, 20, 20]), pa.DEV_BAD_LEN),
                        (dict(lens=[20, 3, 20, 20]), pa.DEV_BAD_LEN), (dict(start=[0, 8, 4, 12, 16]), pa.DEV_BAD_LEN),
                        (dict(start=[0, 4, 8, 12, 99]), pa.DEV_BAD_LEN), (dict(block=1), pa.DEV_BAD_BLOCK)):
        lens = torch.tensor(change.get("lens", [20] * 4), dtype=torch.int32)
        st = torch.tensor(change.get("start", start.tolist()), dtype=torch.int32)
        tab = c.tab.clone()
        if "block" in change:
            tab[1, 1] = -5
        good = [b for b in range(4) if st[b] >= 0 and st[b] <= st[b + 1] <= 16 and 0 <= st[b + 1] - st[b] <= lens[b] <= 64
                and not ("block" in change and b == 1)]
        got = [x.cuda() for x in (c.k, c.v, c.ks, c.vs)]
        pa.append_fp8_blocks(key.cuda(), val.cuda(), st.cuda(), tab.cuda(), lens.cuda(), *got)
        assert pa.last_error() == bit
        ref = [x.numpy() for x in (c.k, c.v, c.ks, c.vs)]
        for b in good:
            r0, r1 = int(st[b]), int(st[b + 1])
            ref = oracle.append_fp8_blocks(key[r0:r1].double().numpy(), val[r0:r1].double().numpy(), [0, r1 - r0],
                                           tab[b:b + 1].numpy(), lens[b:b + 1].numpy(), *ref)
        for g, r in zip(got, ref):
            assert np.array_equal(g.cpu().numpy(), r)


def test_copy_on_write(pa):
    c = Case("e4m3", [40, 30], 6, 6, 64, 16)
    pairs = torch.tensor([[int(c.tab[0, 0]), int(c.tab[1, 1])], [int(c.tab[0, 1]), int(c.tab[0, 2])]])
    got = [x.cuda() for x in (c.k, c.v, c.ks, c.vs)]
    pa.copy_blocks_fp8_blocks(*got, pairs.cuda())
    assert pa.last_error() == 0
    for g, x in zip(got, (c.k, c.v, c.ks, c.vs)):
        r = x.clone()
        for s, d in pairs.tolist():
            r[d] = x[s]
        assert torch.equal(g.cpu(), r)


# ------------------------------------------------------------------ decode

LENS = [1, 0, 15, 16, 17, 300, 700, 129, 128]


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 8, 128, 16), (8, 2, 128, 16), (32, 8, 128, 16), (16, 4, 64, 8), (12, 4, 128, 16),
                                         (4, 4, 32, 4), (14, 2, 128, 32), (16, 1, 128, 8), (6, 3, 128, 8), (5, 5, 64, 32),
                                         (64, 2, 128, 16), (8, 1, 128, 4), (7, 1, 128, 16), (24, 3, 64, 16), (18, 2, 128, 16),
                                         (8, 8, 64, 16), (4, 2, 64, 32), (12, 12, 32, 8), (20, 4, 32, 16), (40, 4, 64, 16),
                                         (4, 4, 32, 16), (6, 2, 64, 16)])
@pytest.mark.parametrize("partition", [0, 64, -1])
def test_decode(pa, Hq, Hkv, D, bs, partition):
    c = Case("e4m3", LENS, Hq, Hkv, D, bs, seed=Hq + bs)
    ref, tol = reference(c)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale, partition_size=partition)
    assert pa.last_error() == 0
    check(out, ref, tol)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 128), (4, 2, 64)])
def test_decode_scales_far_apart_and_zero(pa, Hq, Hkv, D):
    c = Case("e4m3", [260, 17, 400], Hq, Hkv, D, 16, seed=4)
    c.vs[c.tab[0, :6].long()] *= 2.0 ** 20
    c.vs[c.tab[0, 6:10].long()] *= 2.0 ** -20
    c.vs[c.tab[2, 3].long()] = 0.0
    c.ks[c.tab[2, 5].long()] = 0.0
    c.ks[c.tab[1, :2].long()] *= 8.0                 # sharp softmax
    ref, tol = reference(c)
    c.cuda()
    out = torch.empty_like(c.q)
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


def test_decode_bad_block_and_length(pa):
    c = Case("e4m3", [100, 100, 100], 8, 2, 128, 16).cuda()
    c.lens[1] = 10 ** 6
    c.tab[2, 2] = -1
    out = torch.empty_like(c.q)
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == pa.DEV_BAD_BLOCK | pa.DEV_BAD_LEN


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64), (8, 4, 32), (3, 3, 64)])
def test_decode_nan_stays_in_its_head(pa, Hq, Hkv, D):
    """A NaN key makes NaN of its own KV head's query heads, a NaN value of its own dim, and of nothing else."""
    c = Case("e4m3", [150, 40], Hq, Hkv, D, 16, seed=6)
    ref, tol = reference(c)
    c.k[c.tab[0, 1].long(), 3, 1, 5] = 0x7F
    c.v[c.tab[1, 0].long(), 2, 0, 7] = 0xFF
    c.cuda()
    out = torch.empty_like(c.q)
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    G = Hq // Hkv
    nan = torch.zeros(out.shape, dtype=torch.bool)
    nan[0, G:2 * G] = True
    nan[1, :G, 7] = True
    assert torch.equal(out.isnan().cpu(), nan)
    check(torch.where(nan.cuda(), torch.zeros_like(out), out), np.where(nan.numpy(), 0, ref), tol)


def test_decode_many_sequences(pa):
    """More sequences than the dense item tables hold."""
    rng = np.random.default_rng(0)
    c = Case("e4m3", rng.integers(0, 40, 1100), 4, 2, 128, 16, seed=1)
    ref, tol = reference(c)
    c.cuda()
    out = torch.empty_like(c.q)
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


# ------------------------------------------------------------------ causal attention of the newest tokens

@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (4, 4, 128, 8), (16, 1, 128, 32), (6, 2, 128, 16), (8, 4, 64, 16),
                                         (4, 2, 32, 8), (8, 2, 128, 4), (2, 1, 128, 16), (16, 2, 128, 16), (20, 1, 128, 16)])
def test_prefill(pa, Hq, Hkv, D, bs):
    lens, n = [1, 200, 64, 65, 130, 7, 150], [1, 130, 64, 1, 33, 0, 9]
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=Hq + D, rows=sum(n))
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


def test_prefill_rows_before_the_context_and_rows_past_the_last_sequence(pa):
    c = Case("e4m3", [40, 5], 8, 2, 128, 16, seed=9, rows=30)
    start = torch.tensor([0, 10, 22], dtype=torch.int32)      # 12 rows on a context of 5; rows 22..29 are nobody's
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.full_like(c.q, 7.0)
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out[:22], ref[:22], tol[:22])
    assert (out[10:17] == 0).all() and (out[22:] == 7.0).all()


@pytest.mark.parametrize("start", [[0, 8, 4, 12], [0, 4, 8, 99], [-3, 4, 8, 12]])
def test_prefill_bad_rows(pa, start):
    c = Case("e4m3", [20, 20, 20], 8, 2, 128, 16, rows=12)
    st = torch.tensor(start, dtype=torch.int32)
    c.cuda()
    out = torch.full_like(c.q, 7.0)
    pa.prefill_fp8_blocks(out, c.q, st.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == pa.DEV_BAD_LEN
    bad = [b for b in range(3) if not 0 <= start[b] <= start[b + 1] <= 12]
    for b in bad:
        lo, hi = max(0, start[b]), min(12, start[b + 1])
        owned = set(range(lo, hi)) - {r for g in range(3) if g not in bad for r in range(start[g], start[g + 1])}
        assert all((out[r] == 7.0).all() for r in owned)
