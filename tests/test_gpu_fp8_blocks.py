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


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (16, 1, 128, 8), (4, 2, 64, 16), (8, 4, 32, 32), (4, 2, 128, 4)])
@pytest.mark.parametrize("first", [True, False])
def test_decode_looks_at_values_of_small_scale(pa, Hq, Hkv, D, bs, first):
    """The softmax sits on blocks whose V scale is 2^-24 of the others': their digits are kept.  A token's
    product of weight and V scale is off by 2^-8 of itself, or by 2^-19 of the head's largest."""
    L = 420
    c = Case("e4m3", [L], Hq, Hkv, D, bs, seed=bs, spare_cols=0)
    mine = np.zeros(L, dtype=bool)
    mine[:64] = first
    mine[320:384] = not first
    blocks = c.tab[0, [j for j in range(-(-L // bs)) if mine[j * bs]]].long()
    c.vs[blocks] *= 2.0 ** -24
    G = Hq // Hkv
    for h in range(Hkv):                             # the group's queries agree, and those blocks' keys with them
        c.q[0, h * G:(h + 1) * G] = c.q[0, h * G]
        c.k[blocks, :, h] = (c.q[0, h * G] * 64).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
    c.ks[:] = 2.0 ** -2
    K, V = c.f64_pools()
    q = c.q.double().numpy()
    at = [(int(c.tab[0, t // bs]), t % bs) for t in range(L)]
    ref, tol = np.zeros(c.q.shape), np.zeros(c.q.shape)
    for h in range(Hq):
        k, v = (np.stack([x[b, i, h // G] for b, i in at]) for x in (K, V))
        vs = np.array([float(c.vs[b, h // G]) for b, _ in at])
        s = k @ q[0, h] * c.scale
        p = np.exp(s - s.max())
        p /= p.sum()
        assert p[~mine].max() < 2.0 ** -34           # (with their scales they are still the smaller products)
        ref[0, h] = p @ v
        ds = np.abs(k * q[0, h]).sum(1).max() * c.scale * ((D + 4) * 2.0 ** -24 + 2.0 ** -20)
        A = p @ np.abs(v)
        tol[0, h] = (2.0 ** -9 * np.abs(ref[0, h]) + (2.0 ** -8 + np.expm1(2 * ds) + (L + 64) * 2.0 ** -23) * A +
                     2.0 ** -19 * (p * vs).max() * np.abs(v / vs[:, None]).sum(0))
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


@pytest.mark.parametrize("B", [128, 129, 300])
def test_prefill_many_sequences(pa, B):
    """Batches on both sides of the size up to which the longest contexts come first."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1, 150, B)
    n = np.minimum(lens, rng.choice([0, 1, 1, 1, 2, 33, 70], B))
    c = Case("e4m3", lens, 8, 2, 128, 16, seed=B, rows=int(n.sum()))
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


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (4, 4, 128, 8), (8, 4, 64, 16), (4, 2, 128, 4)])
def test_prefill_nan_reaches_the_rows_that_see_it(pa, Hq, Hkv, D, bs):
    """A NaN value makes NaN of its dim in the rows at and past it, a NaN key of those rows' whole heads; rows
    before them, in the same tile of keys or of queries, keep their numbers."""
    lens, n = [300, 90], [300, 40]
    c = Case("e4m3", lens, Hq, Hkv, D, bs, seed=5, rows=sum(n))
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    nan = np.zeros(c.q.shape, dtype=bool)
    G = Hq // Hkv
    for x, b, t, h, d in ((c.v, 0, 77, 1, 3), (c.v, 0, 200, 1, 3), (c.v, 0, 70, 1, 9), (c.v, 0, 299, 0, D - 1),
                          (c.v, 1, 60, 0, 0), (c.k, 0, 130, 0, 5), (c.k, 1, 89, 1, 1)):
        x[int(c.tab[b, t // bs]), t % bs, h, d] = 0xFF if t & 1 else 0x7F
        row = int(start[b]) + max(0, t - (lens[b] - n[b]))
        nan[row:int(start[b + 1]), h * G:(h + 1) * G, d if x is c.v else slice(None)] = True
    c.cuda()
    out = torch.empty_like(c.q)
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    assert np.array_equal(out.isnan().cpu().numpy(), nan)
    check(torch.where(torch.from_numpy(nan).cuda(), torch.zeros_like(out), out), np.where(nan, 0, ref), tol)


@pytest.mark.parametrize("power", [-20, -60, -120])
def test_prefill_small_queries_and_blocks_of_zeros(pa, power):
    """Scores far below 1 next to masked ones: the causal mask stays a mask."""
    lens, n = [200, 70], [200, 3]
    c = Case("e4m3", lens, 8, 2, 128, 16, seed=8, rows=sum(n))
    c.q *= 2.0 ** power
    for j in (0, 3, 12):
        c.ks[c.tab[0, j].long()] = 0.0
        c.k[c.tab[0, j].long()] = 0
    c.ks[c.tab[1, :4].long()] = 2.0 ** -100
    start = _start(n)
    ref, tol = reference(c, start.numpy())
    c.cuda()
    out = torch.empty_like(c.q)
    pa.prefill_fp8_blocks(out, c.q, start.cuda(), c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)


def test_decode_on_another_stream_keeps_its_own_workspace(pa):
    """A call that makes its workspace and runs on a stream that is not the current one: what the current stream
    allocates and writes next is other memory."""
    c = Case("e4m3", [9000] * 8, 8, 2, 128, 16, seed=2)
    ref, tol = reference(c)
    c.cuda()
    out = torch.empty_like(c.q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    n = pa.alloc_fp8_blocks_workspace(c.q, c.k, c.tab).numel()
    assert n > 16
    for _ in range(20):
        pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale, stream=side)
        torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert pa.last_error() == 0
    check(out, ref, tol)
