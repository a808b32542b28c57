"""Ragged causal attention over expanded latent vectors on the GPU against the oracle."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import f64
from _latent import check, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _run(pa, q, start, kv, key, kv_start, scale, Dv, **kw):
    out = torch.full((q.shape[0], q.shape[1], Dv), float("nan"), dtype=q.dtype, device="cuda")
    assert pa.latent_prefill(out, q, _i32(start), kv, key, _i32(kv_start), scale, **kw) is out
    return out


def _case(lens, new, H, Dk, P, Dv, seed=0, wide=0):
    start, kv_start = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(lens)])
    T = int(kv_start[-1])
    return (randn(seed, int(start[-1]), H, Dk + P), start, randn(seed + 1, T, H, Dk + Dv),
            randn(seed + 2, T, wide + P)[:, wide:], kv_start, (Dk + P) ** -0.5)


def _want(q, start, kv, key, kv_start, scale):
    return oracle.latent_prefill(f64(q), start, f64(kv), f64(key), kv_start, scale)


@pytest.mark.parametrize("Dk,P,Dv", [(128, 64, 128), (64, 32, 64), (128, 32, 64), (32, 16, 128), (64, 64, 32), (128, 48, 128)])
@pytest.mark.parametrize("H,lens,new", [(1, [1], [1]), (3, [5, 130, 64], [5, 1, 64]), (2, [300, 129], [257, 129]), (5, [40, 700], [0, 3]),
                                        (1, [260, 513], [130, 300])])
def test_ragged(pa, Dk, P, Dv, H, lens, new):
    a = _case(lens, new, H, Dk, P, Dv, seed=H)
    check(_run(pa, *a, Dv), *_want(*a))
    assert pa.last_error() == 0


@pytest.mark.parametrize("Dk,P,Dv", [(128, 64, 128), (64, 32, 32), (32, 48, 64)])
def test_many_heads(pa, Dk, P, Dv):
    """More (256 rows, head) pairs than the GPU takes at a time: two row tiles a CTA, several items each."""
    a = _case([300, 129, 520, 7, 0, 260], [257, 129, 400, 9, 0, 4], 90, Dk, P, Dv, seed=3)
    check(_run(pa, *a, Dv), *_want(*a))
    assert pa.last_error() == 0


def test_whole_prompt_of_many_tiles(pa):
    a = _case([1500, 1100], [1500, 1100], 34, 128, 64, 128, seed=5)
    check(_run(pa, *a, 128), *_want(*a))
    assert pa.last_error() == 0


def test_many_short_sequences(pa):
    lens = [(7 * i) % 31 + 1 for i in range(150)]
    new = [(5 * i) % (L + 1) for i, L in enumerate(lens)]
    a = _case(lens, new, 2, 128, 64, 128)
    check(_run(pa, *a, 128), *_want(*a))
    assert pa.last_error() == 0


def test_strided_shared_keys(pa):
    """The shared keys as a view behind the latent vectors, as rows taken back from a cache have them."""
    a = _case([90, 200], [90, 50], 4, 128, 64, 128, wide=512)
    assert a[3].stride(0) == 576
    check(_run(pa, *a, 128), *_want(*a))


@pytest.mark.parametrize("factor", [8.0, 60.0])
@pytest.mark.parametrize("H", [2, 120])
def test_scores_far_apart(pa, factor, H):
    q, start, kv, key, kv_start, scale = _case([700], [700], H, 128, 64, 128, seed=4)
    for j in range(0, 700, 64):                               # growing keys: the maximum moves in every tile
        kv[j:j + 64, :, :128] *= 1.0 + j / 64
    a = (q, start, kv, key, kv_start, scale * factor)
    check(_run(pa, *a, 128), *_want(*a))
    a = (torch.zeros_like(q), start, kv, key, kv_start, 1.0)
    check(_run(pa, *a, 128), *_want(*a))


def test_rows_with_nothing_to_see(pa):
    """More rows than context, a context of zero, rows behind the last sequence, sequences without rows."""
    for H in (3, 70):
        _nothing_to_see(pa, H)


def _nothing_to_see(pa, H):
    q, kv, key = randn(1, 200, H, 192), randn(2, 170, H, 256), randn(3, 170, 64)
    start, kv_start = np.array([0, 140, 143, 143, 150]), np.array([0, 10, 10, 150, 160])
    want = oracle.latent_prefill(f64(q), start, f64(kv), f64(key), kv_start, 0.07)
    out = _run(pa, q, start, kv, key, kv_start, 0.07, 128)
    check(out, *want)
    assert not out[:130].any() and not out[140:143].any() and torch.isnan(out[150:]).all()
    assert pa.last_error() == 0


@pytest.mark.parametrize("H", [2, 160])                     # a row tile a CTA, and two
def test_nan_stays_with_the_rows_that_see_it(pa, H):
    q, start, kv, key, kv_start, scale = _case([200, 90], [200, 90], H, 128, 64, 128)
    want = _want(q, start, kv, key, kv_start, scale)
    kv[150, 1, 200] = float("nan")                            # a value: its element from row 150 on
    key[180] = float("nan")                                   # a shared key: every head from row 180 on
    kv2 = torch.cat([kv, torch.full_like(kv[:64], float("nan"))])       # and rows that no sequence has
    key2 = torch.cat([key, torch.full_like(key[:64], float("nan"))])
    out = _run(pa, q, start, kv2, key2, kv_start, scale, 128)
    rows = list(range(150)) + list(range(200, 290))
    check(out[rows], *(x[rows] for x in want))
    assert torch.isnan(out[180:200]).all() and torch.isnan(out[150:180, 1, 200 - 128]).all()
    mid = list(range(150, 180))
    got, (w, m, s) = out[mid], (x[mid] for x in want)
    w[:, 1, 72] = np.nan
    check(got, w, m, s)


@pytest.mark.parametrize("H", [2, 160])
def test_rows_before_the_context_beside_a_nan(pa, H):
    """More rows than context: the rows that see nothing are zeros, whatever the values hold."""
    q, kv, key = randn(1, 140, H, 192), randn(2, 20, H, 256), randn(3, 20, 64)
    kv[0, :, 130] = float("nan")
    start, kv_start = [0, 140], [0, 20]
    out = _run(pa, q, start, kv, key, kv_start, 0.07, 128)
    assert not out[:120].any() and torch.isnan(out[120:, :, 2]).all()
    w, m, s = oracle.latent_prefill(f64(q), start, f64(kv), f64(key), kv_start, 0.07)
    keep = [d for d in range(128) if d != 2]
    check(out[..., keep], w[..., keep], m[..., keep], s)
    assert pa.last_error() == 0


@pytest.mark.parametrize("H", [2, 160])
def test_tokens_of_no_weight_before_low_scores(pa, H):
    """Scores of -inf in whole tiles at the start, then scores far below zero: as if the context began there."""
    for L, hidden, n in ((300, 128, 140), (700, 384, 260), (150, 140, 5)):
        q, start, kv, key, kv_start, _ = _case([L], [n], H, 128, 32, 64, seed=L)
        q[:, :, 150], q[:, :, 151] = 8.0, 1.0
        key[:, 22], key[:hidden, 23] = -50.0, -float("inf")   # every score 400 lower
        want = _want(q, start, kv[hidden:], key[hidden:], [0, L - hidden], 0.5)
        check(_run(pa, q, start, kv, key, kv_start, 0.5, 64), *want)
    assert pa.last_error() == 0


def test_two_calls_at_once(pa):
    """Calls on two streams share nothing."""
    a, b = _case([600, 90], [600, 40], 12, 128, 64, 128, seed=1), _case([333], [333], 40, 64, 32, 64, seed=2)
    one, two = _run(pa, *a, 128), _run(pa, *b, 64)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for st in (s, t):
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        outs.append((_run(pa, *a, 128, stream=s), _run(pa, *b, 64, stream=t)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, one) and torch.equal(y, two) for x, y in outs) and pa.last_error() == 0


def test_bad_starts(pa):
    a = _case([50, 60, 70], [10, 20, 30], 2, 128, 64, 128)
    q, start, kv, key, kv_start, scale = a
    want = _want(*a)
    for st, ks in (([0, 10, 5, 60], kv_start), (start, [0, 50, 40, 180]), ([0, 10, 30, 61], kv_start), (start, [0, 50, 110, 181]),
                   ([-1, 10, 30, 60], kv_start)):
        out = _run(pa, q, st, kv, key, ks, scale, 128)
        assert pa.last_error() == pa.DEV_BAD_LEN
        fit = [b for b in range(3) if 0 <= st[b] <= st[b + 1] <= 60 and 0 <= ks[b] <= ks[b + 1] <= 180]
        for b in fit:
            if st[b] == start[b] and st[b + 1] == start[b + 1] and ks[b] == kv_start[b] and ks[b + 1] == kv_start[b + 1]:
                # (a row of two sequences has no value)
                mine = [i for i in range(start[b], start[b + 1]) if sum(st[x] <= i < st[x + 1] for x in fit) == 1]
                check(out[mine], *(x[mine] for x in want))


def test_same_bits_again_on_another_stream_and_in_a_graph(pa):
    a = _case([300, 170], [300, 20], 4, 128, 64, 128)
    first = _run(pa, *a, 128)
    assert torch.equal(first, _run(pa, *a, 128))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _run(pa, *a, 128, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    q, start, kv, key, kv_start, scale = a
    st, ks = _i32(start), _i32(kv_start)
    out = torch.zeros_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.latent_prefill(out, q, st, kv, key, ks, scale)
    for seed, s2, k2 in ((1, start, kv_start), (2, [0, 5, 320], [0, 100, 470])):
        q.copy_(randn(seed, *q.shape))
        st.copy_(_i32(s2)), ks.copy_(_i32(k2))
        g.replay()
        check(out, *oracle.latent_prefill(f64(q), s2, f64(kv), f64(key), k2, scale))
    assert pa.last_error() == 0
