"""Pins for the oracle of the rotary positions and of latent attention, and pa_rope_steps against it (CPU only)."""

import math

import numpy as np
import pytest

import oracle
from paged_kv_cache_307_gb300 import build as B


@pytest.fixture(scope="module")
def pa():
    B.build()
    from paged_kv_cache_307_gb300 import _lib
    return _lib


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=32.0, original_len=4096.0),
            dict(scaling="yarn", factor=2.5, original_len=100.0, beta_fast=8.0, beta_slow=2.0)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("d,base", [(16, 10000.0), (64, 10000.0), (128, 500000.0), (32, 1.5)])
def test_steps_are_the_frequencies_as_fractions_of_a_turn(pa, kw, d, base):
    f, amp = oracle.rope_frequencies(d, base, **kw)
    steps, a = pa.rope_steps(d, base, **kw)
    assert steps.shape == (d // 2,) and a == np.float32(amp)
    got = steps.numpy().view(np.uint64).astype(object)
    for g, x in zip(got, f):
        # pow and the quotient by 2 pi round in 53 bits each, on either side
        assert abs(int(g) / 2 ** 64 - x / (2 * math.pi)) <= x * 2.0 ** -50 + 2.0 ** -65


def test_scalings_leave_what_they_say():
    f0, _ = oracle.rope_frequencies(64, 10000.0)
    f, amp = oracle.rope_frequencies(64, 10000.0, "yarn", 16.0, 4096.0)
    turns = 4096 * f0 / (2 * math.pi)
    fast, slow = turns >= 64, turns <= 0.5                       # well outside the ramp
    assert fast.any() and slow.any() and amp == 0.1 * math.log(16) + 1
    assert np.allclose(f[fast], f0[fast], rtol=1e-12) and np.allclose(f[slow], f0[slow] / 16, rtol=1e-12)
    assert (np.diff(f / f0) <= 1e-15).all()
    g, _ = oracle.rope_frequencies(64, 10000.0, "ntk", 16.0)
    assert g[0] == 1 and math.isclose(g[-1], f0[-1] / 16, rel_tol=1e-12)     # the slowest pair is interpolated


def test_rotation_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(0)
    f, _ = oracle.rope_frequencies(32, 10000.0)
    x, y = rng.standard_normal((2, 1, 1, 32))
    for layout in ("half", "interleaved"):
        turn = lambda v, p: oracle.rope(v, [p], f, layout=layout)      # noqa: E731
        assert np.allclose(np.linalg.norm(turn(x, 1234)), np.linalg.norm(x))
        assert np.allclose((turn(x, 900) * turn(y, 893)).sum(), (turn(x, 7) * turn(y, 0)).sum())
    half, inter = oracle.rope(x, [5], f), oracle.rope(x.reshape(1, 1, 2, 16).swapaxes(2, 3).reshape(1, 1, 32), [5], f,
                                                      layout="interleaved")
    assert np.allclose(half.reshape(2, 16).T.reshape(-1), inter.reshape(-1))


def test_absorbed_and_expanded_forms_agree():
    """Keys and values multiplied out of the latent vectors, or the products moved to the query and the output."""
    rng = np.random.default_rng(1)
    R, P, Dn, Dv, H, bs = 8, 4, 6, 5, 3, 4
    lens, new = [7, 3, 10], [2, 3, 1]
    start, kv_start = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(lens)])
    cache = rng.standard_normal((9, bs, R + P))
    table = rng.permutation(9).reshape(3, 3)
    up_k, up_v = rng.standard_normal((H, R, Dn)), rng.standard_normal((H, R, Dv))
    q = rng.standard_normal((6, H, Dn + P))
    rows = np.concatenate([cache[table[b]].reshape(-1, R + P)[:n] for b, n in enumerate(lens)])
    kv = np.concatenate([np.einsum("tr,hrd->thd", rows[:, :R], up_k), np.einsum("tr,hrd->thd", rows[:, :R], up_v)], 2)
    want, _, _ = oracle.latent_prefill(q, start, kv, rows[:, R:], kv_start, 0.4)
    qa = np.concatenate([np.einsum("nhd,hrd->nhr", q[..., :Dn], up_k), q[..., Dn:]], 2)
    got, _, _ = oracle.latent_decode(qa, cache, table, lens, 0.4, R, start)
    assert np.allclose(np.einsum("nhr,hrd->nhd", got, up_v), want)
    # one row a sequence is the last of each; a row before the context is zeros
    last, _, _ = oracle.latent_decode(qa[start[1:] - 1], cache, table, lens, 0.4, R)
    assert np.allclose(last, got[start[1:] - 1])
    none, _, _ = oracle.latent_decode(qa[:2], cache, table[:1], [1], 0.4, R, [0, 2])
    assert not none[0].any() and np.allclose(none[1], cache[table[0, 0], 0, :R])
