"""Pins for the oracle of the block-scaled cache, the attention weights and the eviction (CPU only)."""

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("a,s", [(448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                 (1.7500001, 2.0 ** -7), (0.0, 0.0), (1e-40, 2.0 ** -100), (3e38, 2.0 ** 120)])
def test_scale_is_the_smallest_power_of_two(a, s):
    assert oracle.pow2_scale(a) == s
    if s > 2.0 ** -100:
        assert a <= 448 * s and a > 448 * s / 2


def _append_all(x, splits, bs=4, NB=6):
    H, D = x.shape[1:]
    k = np.zeros((NB, bs, H, D), np.uint8)
    sc = np.zeros((NB, 4), np.float32)
    tab = np.array([[3, 1, 5, 0]])
    done = 0
    v, vs = k.copy(), sc.copy()
    for n in splits:
        k, v, sc, vs = oracle.append_fp8_blocks(x[done:done + n], x[done:done + n], [0, n], tab, [done + n], k, v, sc, vs)
        done += n
    return k, sc


def test_append_token_by_token_equals_at_once_for_normal_codes():
    rng = np.random.default_rng(0)
    # magnitudes within the 2**14 range that keeps every rescaled code normal
    x = rng.choice([-1, 1], (14, 3, 8)) * np.exp2(rng.uniform(-3, 3, (14, 3, 8)))
    once, s1 = _append_all(x, [14])
    steps, s2 = _append_all(x, [1] * 14)
    mixed, s3 = _append_all(x, [3, 6, 1, 4])
    assert np.array_equal(s1, s2) and np.array_equal(s1, s3)
    assert np.array_equal(once, steps) and np.array_equal(once, mixed)
    deq = oracle.dequantize_blocks(once, s1)
    got = np.concatenate([deq[3], deq[1], deq[5], deq[0]])[:14]
    assert np.max(np.abs(got - x) / np.abs(x)) <= 2.0 ** -4


def test_append_starts_a_block_afresh_and_keeps_zero_blocks():
    k = np.full((2, 4, 1, 8), 0x7E, np.uint8)
    sc = np.full((2, 4), 64.0, np.float32)
    x = np.zeros((2, 1, 8))
    k2, _, s2, _ = oracle.append_fp8_blocks(x, x, [0, 2], np.array([[1]]), [2], k, k, sc, sc)
    assert s2[1, 0] == 0 and not k2[1, :2].any() and s2[0, 0] == 64 and (k2[0] == 0x7E).all()


def test_weights_sum_to_the_query_heads_and_give_the_output():
    rng = np.random.default_rng(1)
    K, V = rng.standard_normal((2, 5, 4, 2, 8))
    q = rng.standard_normal((1, 6, 8))
    tab = np.array([[4, 0, 2]])
    w = oracle.attention_weights(q, K, tab, [10], 0.3)[0]
    assert np.allclose(w.sum(1), 3)
    out = oracle.paged_decode(q, K, V, tab, [10], 0.3)[0]
    Vr = V[tab[0]].reshape(-1, 2, 8)[:10]
    for g in range(2):
        assert np.allclose(out[3 * g:3 * g + 3].sum(0), w[g] @ Vr[:, g])


def _evict_case(L, budget, recent, sinks, seed=0, kept=0, B=2, H=2, bs=4, D=4, spread=3):
    rng = np.random.default_rng(seed)
    n = -(-L // bs)
    k, v = rng.standard_normal((2, B * n + 2, bs, H, D))
    tab = rng.permutation(B * n + 2)[:B * n].reshape(B, n)
    w = rng.integers(0, spread, (B, H, n * bs)).astype(np.float32)       # many ties
    pos = np.sort(rng.permutation(500)[:n * bs])
    pos = np.broadcast_to(pos, (B, H, n * bs)).astype(np.int32)
    seen = np.full(B, 600 if kept else L)
    return k, v, tab, np.full(B, L), np.full(B, kept), seen, w, pos, budget, recent, sinks


@pytest.mark.parametrize("L,budget,recent,sinks,kept", [(13, 7, 2, 1, 0), (13, 13, 0, 0, 0), (5, 9, 3, 2, 0),
                                                        (16, 8, 8, 0, 0), (15, 1, 1, 0, 0), (15, 6, 2, 2, 6)])
def test_evict_keeps_the_best_and_carries_them(L, budget, recent, sinks, kept):
    c = _evict_case(L, budget, recent, sinks, kept=kept)
    k, v, tab, lens, _, seen, w, pos, *_ = c
    k2, v2, _, _, new, w2, p2 = oracle.evict(*c)
    assert (new == min(L, budget)).all()
    for b in range(2):
        rows, rows2 = k[tab[b]].reshape(-1, 2, 4), k2[tab[b]].reshape(-1, 2, 4)
        for h in range(2):
            where = np.array([pos[b, h, t] if t < kept else seen[b] - L + t for t in range(L)])
            n = new[b]
            src = [int(np.flatnonzero(where == p)[0]) for p in p2[b, h, :n]]
            assert len(set(src)) == n                                   # no token twice
            assert np.array_equal(rows2[:n, h], rows[src, h])           # its row came with it
            assert np.array_equal(w2[b, h, :n], w[b, h, src])
            assert (w2[b, h, n:] == 0).all() and (p2[b, h, n:] == -1).all()
            must = {t for t in range(L) if where[t] < sinks or where[t] >= seen[b] - recent}
            gone = set(range(L)) - set(src)
            assert n < L or not gone
            assert not gone & must
            rest = [t for t in src if t not in must]
            if gone and rest:
                # nothing dropped outweighs a kept one; of equals the lower slots were kept
                worst = min((w[b, h, t], -t) for t in rest)
                assert all((w[b, h, t], -t) < worst for t in gone)
            assert all(s == t for t, s in enumerate(src) if s < n)      # what could stay stayed


def test_evict_does_not_change_what_attention_sees_of_the_kept():
    c = _evict_case(14, 8, 2, 1, seed=3)
    k, v, tab, lens, _, _, w, pos, *_ = c
    k2, v2, _, _, new, w2, p2 = oracle.evict(*c)
    q = np.random.default_rng(5).standard_normal((2, 2, 4))
    out = oracle.paged_decode(q, k2, v2, tab, new, 0.5)
    for b in range(2):
        for h in range(2):
            keep = np.sort(p2[b, h, :8])
            K, V = k[tab[b]].reshape(-1, 2, 4)[keep, h], v[tab[b]].reshape(-1, 2, 4)[keep, h]
            assert np.allclose(out[b, h], oracle.dense_attention(q[b, h:h + 1], K[:, None], V[:, None], 0.5)[0])


def test_evict_requantises_between_block_scales():
    rng = np.random.default_rng(7)
    codes = oracle.e4m3_encode(rng.standard_normal((5, 4, 1, 8)) * 64)
    sc = np.exp2(rng.integers(-7, -3, (5, 4)).astype(np.float32))
    tab, L = np.array([[2, 0, 4, 1]]), 15
    w = rng.random((1, 1, 16)).astype(np.float32)
    pos = np.full((1, 1, 16), -1, np.int32)
    k2, _, s2, _, new, _, p2 = oracle.evict(codes, codes, tab, [L], [0], [L], w, pos, 6, 1, 1, sc, sc)
    was, now = oracle.dequantize_blocks(codes, sc), oracle.dequantize_blocks(k2, s2)
    was, now = was[tab[0]].reshape(-1, 8), now[tab[0]].reshape(-1, 8)
    for t in range(6):
        x, y = was[p2[0, 0, t]], now[t]
        # a rescaled code is off by at most half a subnormal step of its new scale, or half a step of its value
        assert np.all(np.abs(x - y) <= np.maximum(2.0 ** -10 * s2[tab[0][t // 4], 0], 0))
    assert (s2 >= sc).all()
