"""Rotary positions and attention over latent vectors.  Float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages do not print these operations; this restates the definitions of the
C header one step at a time:

* rotary: pair i of a head is a complex number, multiplied by
  A exp(i p f_i); the frequencies plain, interpolated, with a raised base, or
  interpolated only where a pair turns seldom.
* latent attention: a softmax over a context whose rows are keys and values
  (absorbed), or whose keys are a head's own part and a shared one (expanded);
  row i of a sequence's n newest sits at position L - n + i and sees what is not
  behind it.

Attention returns, beside the output, two sums that bound the error of an
implementation in few bits: sum_t w_t |v_t| of every output element and
max_t sum_d |q_d k_td| of every row.
"""

import math

import numpy as np

from .attention import _as_f64


def rope_frequencies(rotary_dim, base, scaling="none", factor=1.0, original_len=4096.0, beta_fast=32.0,
                     beta_slow=1.0):
    """(frequencies in radians a position, amplitude)"""
    d = rotary_dim
    if scaling == "ntk":
        base = base * factor ** (d / (d - 2))
    f = [base ** (-2 * i / d) for i in range(d // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "yarn":
        return np.array(f), 1.0

    def pair(turns):            # pair i makes original_len base^(-2i/d) / 2 pi turns
        return d * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(0, math.floor(pair(beta_fast))), min(d - 1, math.ceil(pair(beta_slow)))
    part = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(d // 2)]
    return np.array([x * (r / factor + 1 - r) for x, r in zip(f, part)]), 0.1 * math.log(factor) + 1


def rope(x, positions, frequencies, amplitude=1.0, layout="half"):
    """x [N, H, D] with its first 2 len(frequencies) elements rotated."""
    y = np.array(_as_f64(x), copy=True)
    n = len(frequencies)
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    turn = amplitude * np.exp(1j * np.asarray(positions, dtype=np.float64)[:, None, None] * frequencies)
    z = (y[..., a] + 1j * y[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _attend(q, K, V, scale, at):
    """q [n, d], K [L, d], V [L, e], row i seeing 0..at[i]: output, sum w |v|, max sum |q k|."""
    out, mass, size = np.zeros((len(q), V.shape[1])), np.zeros((len(q), V.shape[1])), np.zeros(len(q))
    live = [i for i, p in enumerate(at) if p >= 0]
    if not live:
        return out, mass, size
    if np.isfinite(K).all() and np.isfinite(V).all():
        late = np.arange(len(K))[None] > np.asarray(at)[live][:, None]
        s = np.where(late, -np.inf, scale * (q[live] @ K.T))
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[live], mass[live] = w @ V, w @ np.abs(V)
        size[live] = scale * np.where(late, 0, np.abs(q[live]) @ np.abs(K).T).max(1)
        return out, mass, size
    for i in live:                       # (a product with 0 would carry a NaN into rows that do not see it)
        n = at[i] + 1
        s = scale * (K[:n] @ q[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        out[i], mass[i] = w @ V[:n], w @ np.abs(V[:n])
        size[i] = scale * (np.abs(K[:n]) @ np.abs(q[i])).max()
    return out, mass, size


def latent_decode(q, cache, block_tables, context_lens, scale, latent_dim, query_start=None):
    """q [rows, H, R + P] over cache [NB, bs, R + P]: out, mass [rows, H, R], size [rows, H].  Rows of no sequence
    are NaN."""
    q, cache = _as_f64(q), _as_f64(cache)
    start = range(len(context_lens) + 1) if query_start is None else query_start
    rows, H, W = q.shape
    out, mass = np.full((2, rows, H, latent_dim), np.nan)
    size = np.full((rows, H), np.nan)
    bs = cache.shape[1]
    for b, L in enumerate(context_lens):
        a, e = int(start[b]), int(start[b + 1])
        C = cache[np.asarray(block_tables[b][:-(-int(L) // bs)], dtype=np.int64)].reshape(-1, W)[:L]
        at = [int(L) - (e - a) + i for i in range(e - a)]
        for h in range(H):
            out[a:e, h], mass[a:e, h], size[a:e, h] = _attend(q[a:e, h], C, C[:, :latent_dim], scale, at)
    return out, mass, size


def latent_prefill(q, query_start, kv, key_rope, kv_start, scale):
    """q [rows, H, Dk + P], kv [T, H, Dk + Dv], key_rope [T, P]: out, mass [rows, H, Dv], size [rows, H]."""
    q, kv, key_rope = _as_f64(q), _as_f64(kv), _as_f64(key_rope)
    rows, H, W = q.shape
    Dk = W - key_rope.shape[1]
    out, mass = np.full((2, rows, H, kv.shape[2] - Dk), np.nan)
    size = np.full((rows, H), np.nan)
    for b in range(len(query_start) - 1):
        a, e, k0, k1 = int(query_start[b]), int(query_start[b + 1]), int(kv_start[b]), int(kv_start[b + 1])
        at = [(k1 - k0) - (e - a) + i for i in range(e - a)]
        for h in range(H):
            K = np.concatenate([kv[k0:k1, h, :Dk], key_rope[k0:k1]], 1)
            out[a:e, h], mass[a:e, h], size[a:e, h] = _attend(q[a:e, h], K, kv[k0:k1, h, Dk:], scale, at)
    return out, mass, size
