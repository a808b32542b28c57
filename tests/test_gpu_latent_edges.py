"""Latent attention on the GPU where values or scores are not finite, against the oracle: who sees them, what the others
keep, and that neither the context's length nor the number of such values holds a call up."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import f64
from _latent import Cache, check, randn

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:.*encountered in.*:RuntimeWarning")]

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _check(got, want, mass, size):
    """What is not finite has to be the same, the rest within its bound."""
    g = f64(got)
    odd = ~np.isfinite(want)
    assert np.array_equal(g[odd], want[odd], equal_nan=True), "%d of %d are not what they should be, first %s" % (
        (~((g[odd] == want[odd]) | (np.isnan(g[odd]) & np.isnan(want[odd])))).sum(), odd.sum(), np.argwhere(odd)[0])
    want = np.where(odd, np.nan, want)
    check(torch.from_numpy(np.where(odd, np.nan, g)), want, mass, size)


def _prefill(pa, q, start, kv, key, kv_start, scale):
    Dv = kv.shape[2] - (q.shape[2] - key.shape[1])
    out = torch.full((q.shape[0], q.shape[1], Dv), 7.0, dtype=q.dtype, device="cuda")
    st, ks = (torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (start, kv_start))
    return pa.latent_prefill(out, q, st, kv, key, ks, scale)


def _prefill_check(pa, *a):
    q, start, kv, key, kv_start, scale = a
    _check(_prefill(pa, *a), *oracle.latent_prefill(f64(q), start, f64(kv), f64(key), kv_start, scale))
    assert pa.last_error() == 0


# ------------------------------------------------------------------ expanded

@pytest.mark.parametrize("Dk,P,Dv", [(32, 16, 32), (128, 64, 128), (64, 32, 64)])
@pytest.mark.parametrize("H", [2, 160])                     # a row tile a CTA, and two
def test_values_that_are_not_finite(pa, H, Dk, P, Dv):
    """Infinities and NaN in tokens that no new row, some or all new rows see, several in one element."""
    lens, new = [300, 60, 131], [290, 3, 131]
    start, kv_start = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(lens)])
    q, kv, key = randn(1, start[-1], H, Dk + P), randn(2, kv_start[-1], H, Dk + Dv), randn(3, kv_start[-1], P)
    for t, d, x in ((0, 0, INF), (5, 1, NAN), (9, 2, -INF), (15, 3, INF), (137, 3, -INF), (137, 4, INF), (138, 5, -INF),
                    (200, 4, INF), (255, 6, NAN), (256, 7, INF), (265, 8, -INF), (298, 9, INF), (299, 10, NAN),
                    (300, 11, INF), (357, 12, -INF), (358, 13, NAN), (360, 14, INF), (488, 15, INF), (490, 16, NAN)):
        kv[t, H // 2, Dk + d] = x
    kv[[20, 280], 0, Dk + 20:] = INF
    kv[400, 1] = NAN                                        # keys too: its rows from there on whole
    _prefill_check(pa, q, start, kv, key, kv_start, (Dk + P) ** -0.5)


@pytest.mark.parametrize("H", [3, 48])
def test_many_short_sequences_with_values_that_are_not_finite(pa, H):
    """More items a CTA than are under way at a time, every other one with such a value."""
    lens = [(29 * i) % 150 + 1 for i in range(90)]
    new = [max(1, L // (1 + i % 3)) for i, L in enumerate(lens)]
    start, kv_start = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(lens)])
    q, kv, key = randn(4, start[-1], H, 48), randn(5, kv_start[-1], H, 64), randn(6, kv_start[-1], 16)
    rng = np.random.default_rng(0)
    for b in range(0, 90, 2):
        for _ in range(3):
            kv[kv_start[b] + rng.integers(lens[b]), rng.integers(H), 32 + rng.integers(32)] = rng.choice([INF, -INF, NAN])
    _prefill_check(pa, q, start, kv, key, kv_start, 0.15)


def test_long_contexts_beside_values_that_are_not_finite(pa):
    """A NaN among the newest of 100 000 tokens and an infinity in the first, other sequences and heads beside them:
    nothing waits for rows that are done one by one."""
    lens, new = [100000, 900, 40000], [260, 300, 5]
    H, Dk, P, Dv = 4, 32, 16, 32
    start, kv_start = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(lens)])
    q, kv, key = randn(1, start[-1], H, Dk + P), randn(2, kv_start[-1], H, Dk + Dv), randn(3, kv_start[-1], P)
    scale = 2.0 * (Dk + P) ** -0.5
    out0 = _prefill(pa, q, start, kv, key, kv_start, scale)
    kv[100000 - 30, :, Dk + 3] = NAN
    kv[0, 1, Dk + 5] = INF
    kv[100900, 2, Dk + 6] = INF
    out = _prefill(pa, q, start, kv, key, kv_start, scale)
    assert pa.last_error() == 0
    want = out0.clone()
    want[230:260, :, 3] = NAN
    want[:260, 1, 5] = INF
    want[560:, 2, 6] = INF
    same = (out == want) | (torch.isnan(out) & torch.isnan(want))
    assert same.all(), torch.argwhere(~same)[:5].tolist()
    kv = randn(2, kv_start[-1], H, Dk + Dv)                  # some rows of the finite call against the oracle
    for r in (0, 100, 229, 230, 259, 400, 560, 564):
        b = int(np.searchsorted(start, r, "right")) - 1
        n = int(lens[b] - (start[b + 1] - r) + 1)
        k0 = int(kv_start[b])
        _check(out0[r:r + 1], *oracle.latent_prefill(f64(q[r:r + 1]), [0, 1], f64(kv[k0:k0 + n]), f64(key[k0:k0 + n]), [0, n], scale))


def test_every_value_of_a_head_not_finite(pa):
    """One head all NaN, another all infinite: theirs alone."""
    H = 160
    start = kv_start = [0, 700, 760]
    q, kv, key = randn(1, 760, H, 48), randn(2, 760, H, 64), randn(3, 760, 16)
    out0 = _prefill(pa, q, start, kv, key, kv_start, 0.2)
    kv[:, 3, 32:], kv[:700, 7, 32:] = NAN, -INF
    out = _prefill(pa, q, start, kv, key, kv_start, 0.2)
    want = out0.clone()
    want[:, 3], want[:700, 7] = NAN, -INF
    assert ((out == want) | (torch.isnan(out) & torch.isnan(want))).all() and pa.last_error() == 0


@pytest.mark.parametrize("H", [2, 160])
def test_sums_of_large_values(pa, H):
    """Values up to 1e36 under weights that grow from tile to tile: their sums before the division stay finite."""
    L = 300
    q, kv, key = randn(1, L, H, 48), randn(2, L, H, 64), randn(3, L, 16, scale=0.0)
    q[:, :, :48], kv[:, :, 32:] = 0, kv[:, :, 32:].sign() * 1e36
    q[:, :, 47] = 1.0
    key[128:, 15], key[256:, 15] = 5.0, 10.0                # scores of 0, 7.2 and 14.4 in powers of 2
    _prefill_check(pa, q, [0, L], kv, key, [0, L], 1.0)


def test_more_rounds_than_are_told_apart(pa):
    """More than 1024 items a CTA, some of them with a value that is not finite, which the first row of two does not
    see."""
    B, H = 1300, 128
    start = np.arange(B + 1) * 2
    q, kv, key = randn(1, 2 * B, H, 48), randn(2, 2 * B, H, 64), randn(3, 2 * B, 16)
    want = _prefill(pa, q, start, kv, key, start, 0.2)
    rng = np.random.default_rng(1)
    for b, h, d in zip(rng.integers(0, B, 60).tolist(), rng.integers(0, H, 60).tolist(), rng.integers(0, 32, 60).tolist()):
        kv[2 * b + 1, h, 32 + d] = want[2 * b + 1, h, d] = INF
    assert torch.equal(_prefill(pa, q, start, kv, key, start, 0.2), want) and pa.last_error() == 0


def test_contexts_longer_than_the_limit(pa):
    """A context of more than 2^26 tokens writes nothing and is not walked; the one beside it is as ever."""
    L = (1 << 26) + 1
    kv, key = torch.empty(L + 40, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(L + 40, 16, dtype=torch.bfloat16, device="cuda")
    kv[L:], key[L:] = randn(1, 40, 1, 64), randn(2, 40, 16)
    q = randn(3, 10, 1, 48)
    out = _prefill(pa, q, [0, 4, 10], kv, key, [0, L, L + 40], 0.2)
    assert pa.last_error() == pa.DEV_BAD_LEN and (out[:4] == 7.0).all()
    _check(out[4:], *oracle.latent_prefill(f64(q[4:]), [0, 6], f64(kv[L:]), f64(key[L:]), [0, 40], 0.2))


# ------------------------------------------------------------------ absorbed

def _decode(pa, c, q, scale, start=None):
    out = torch.full((*q.shape[:2], c.R), 7.0, dtype=q.dtype, device="cuda")
    st = None if start is None else torch.tensor(np.asarray(start), dtype=torch.int32, device="cuda")
    return pa.latent_decode(out, q, c.cache, c.table, c.lens, scale, query_start=st)


def _put(c, b, t, d, x):
    c.cache[int(c.table[b, t // c.bs]), t % c.bs, d] = x


@pytest.mark.parametrize("R,P", [(256, 32), (512, 64)])
@pytest.mark.parametrize("H,lens,new", [(8, [100, 60], [10, 2]), (40, [300, 129, 50], [4, 4, 1]), (128, [400, 140], [2, 3]),
                                        (16, [128 * 23 + 2, 70], [3, 1]), (1, [700], [150]), (64, [128 * 5 + 1, 128 * 2 + 1], [1, 1])])
def test_infinite_values_under_scores_of_minus_infinity(pa, R, P, H, lens, new):
    """An infinity whose score is -inf: a weight of zero, and NaN in its element, for newest tokens (which some rows do
    not see) as for older ones, and where it is all that a CTA has of a row."""
    c = Cache(lens, R, P, 16, seed=H)
    start = np.concatenate([[0], np.cumsum(new)])
    q = randn(H, int(start[-1]), H, R + P)
    scale = 2.0 * (R + P) ** -0.5
    size = c.oracle(q, scale, start)[2]
    for b, (L, n) in enumerate(zip(lens, new)):
        _put(c, b, L - 1, 70, -INF)                       # for rows of a positive q: -inf, of a negative one: NaN whole
        if n > 1:
            _put(c, b, L - n // 2 - 1, 100, INF)
    q[:, :, 70], q[:, :, 100] = q[:, :, 70].abs(), -q[:, :, 100].abs()
    q[:, H // 2, 70] *= -1
    want, mass, _ = c.oracle(q, scale, start)
    assert np.isnan(want).any() and not np.isnan(want).all(2).all()
    _check(_decode(pa, c, q, scale, None if max(new) == 1 else start), want, mass, size * 1.5)
    assert pa.last_error() == 0


@pytest.mark.parametrize("H,R,bs", [(16, 512, 16), (64, 512, 16), (16, 256, 8), (40, 128, 32)])
def test_last_tiles_of_one_block(pa, H, R, bs):
    """Tiles in which not every copying warp has something to copy, dozens of them a CTA, one after the other and
    between whole ones."""
    B = 2500
    lens = [1 + (7 * b) % bs + (128 if b % 3 == 0 else 0) for b in range(B)]
    c = Cache([256], R, 32, bs)
    q = randn(H, 1, H, R + 32)
    scale = (R + 32) ** -0.5
    want = {}
    for L in set(lens):
        one = Cache([1], R, 32, bs)
        one.cache, one.table, one.lens = c.cache, c.table, torch.tensor([L], dtype=torch.int32, device="cuda")
        want[L] = one.oracle(q, scale)
    c.table, c.lens = c.table.repeat(B, 1), torch.tensor(lens, dtype=torch.int32, device="cuda")
    check(_decode(pa, c, q.repeat(B, 1, 1), scale), *(np.concatenate([want[L][i] for L in lens]) for i in range(3)))
    assert pa.last_error() == 0


@pytest.mark.parametrize("H", [16, 64])
def test_sums_of_large_latent_values(pa, H):
    """Values of 1e36 under weights that grow from tile to tile: their sums before the division stay finite."""
    c = Cache([500], 256, 32, 16)
    ids, sign = c.table[0].long(), c.cache[c.table[0].long(), :, :256].float().nan_to_num().sign()
    c.cache[ids, :, :256] = sign.to(c.cache.dtype) * 1e36
    c.cache[ids, :, 256:] = 0.0
    for j in range(1, 4):                                   # scores of 0, 7.2, 14.4 and 21.6 in powers of 2
        c.cache[ids[8 * j:8 * j + 8], :, 287] = 5.0 * j
    q = torch.zeros(1, H, 288, dtype=torch.bfloat16, device="cuda")
    q[:, :, 287] = 1.0
    want = c.oracle(q, 1.0)
    B = 160
    c.table, c.lens = c.table.repeat(B, 1), c.lens.repeat(B)
    check(_decode(pa, c, q.repeat(B, 1, 1), 1.0), *(x.repeat(B, 0) for x in want))
    assert pa.last_error() == 0


@pytest.mark.parametrize("L", [100, 3000])
def test_rows_of_no_weight_at_all(pa, L):
    """Every score -inf: zeros, whole or cut among CTAs, and nothing of it in other rows."""
    c = Cache([L, 50], 256, 32, 16)
    q = randn(1, 2, 16, 288)
    q[:, :, 281] = 1.0
    want, mass, size = c.oracle(q, 0.1)
    c.cache[c.table[0, :-(-L // 16)].long(), :, 281] = -INF
    want[0], mass[0] = 0, 0
    check(_decode(pa, c, q, 0.1), want, mass, size)
    q, kv, key = randn(1, 210, 2, 192), randn(2, 210, 2, 256), randn(3, 210, 64)
    q[:, :, 191] = 1.0
    st = [0, 150, 210]
    want, mass, size = oracle.latent_prefill(f64(q), st, f64(kv), f64(key), st, 0.07)
    key[:150, 63] = -INF
    want[:150], mass[:150] = 0, 0
    check(_prefill(pa, q, st, kv, key, st, 0.07), want, mass, size)
    assert pa.last_error() == 0


@pytest.mark.parametrize("B", [385, 700, 1500])
@pytest.mark.parametrize("H,new", [(16, False), (3, False), (64, False), (40, True), (128, True)])
def test_more_sequences_than_threads(pa, B, H, new):
    """Several sequences a thread where the batch is cut: empty contexts and sequences without rows among them, cuts at
    any of them."""
    lens = [0 if b % 7 == 3 else (37 * b) % 300 + 1 for b in range(B)]
    rows = [(0, 2, 1, 3, 0)[b % 5] if new else 1 for b in range(B)]
    c = Cache(lens, 128, 16, 16, seed=B)
    start = np.concatenate([[0], np.cumsum(rows)])
    q = randn(H, int(start[-1]), H, 144)
    check(_decode(pa, c, q, 0.15, start if new else None), *c.oracle(q, 0.15, start))
    assert pa.last_error() == 0
