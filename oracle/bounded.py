"""A cache of bounded length: e4m3 blocks with one scale per (block, KV head),
attention weights, and eviction by their running totals.  Float64 / exact.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Layout as in ``attention.py``; scales are [NB, row] with entry h of a row the
scale of KV head h.  The pages do not print these operations; they restate
the definitions of the C header, one step at a time:

* append: for each block and head the new tokens touch, the scale is the
  smallest power of two s with max|x| <= 448 s (at least 2**-100, 0 for
  nothing but zeros), not below the scale of a block that holds earlier tokens
  of the sequence; x / s is encoded, earlier codes are re-encoded.
* weights: softmax weight of every token, summed over the query heads of its
  KV head.
* evict: the budget tokens of a (sequence, KV head) that come first by
  (protected, weight, lower slot) stay; the others' slots below the budget are
  filled, in order, by the kept tokens at or above it.
"""

import math

import numpy as np

from .attention import gather_context, _as_f64
from .quant import e4m3_decode, e4m3_encode

MIN_SCALE = 2.0 ** -100


def pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s, at least 2**-100; 0 for 0."""
    a = float(amax)
    if a == 0:
        return 0.0
    k = math.frexp(a)[1] - 10                 # a >= 2**(k+9) > 448 * 2**k: too small
    while a > 448.0 * math.ldexp(1.0, k):
        k += 1
    return max(math.ldexp(1.0, k), MIN_SCALE)


def dequantize_blocks(codes, scales):
    """Codes [NB, bs, H, D] and scales [NB, >= H] -> float64 values."""
    H = codes.shape[2]
    return e4m3_decode(codes) * np.asarray(scales, dtype=np.float64)[:, None, :H, None]


def _encode_over(x, s):
    """Codes of x / s (NaN -> the NaN code, infinities saturate)."""
    y = np.asarray(x, dtype=np.float64) * ((1.0 / s) if s > 0 else 0.0)
    code = e4m3_encode(np.where(np.isnan(y), 0.0, y))
    return np.where(np.isnan(y), np.uint8(0x7F), code).astype(np.uint8)


def append_fp8_blocks(key, value, query_start, block_tables, context_lens, k_codes, v_codes, k_scale, v_scale):
    """Returns new (k_codes, v_codes, k_scale, v_scale)."""
    outs = [np.array(a, copy=True) for a in (k_codes, v_codes, k_scale, v_scale)]
    bs, H = k_codes.shape[1], k_codes.shape[2]
    for x, codes, scale in ((key, outs[0], outs[2]), (value, outs[1], outs[3])):
        x = _as_f64(x)
        for b in range(len(context_lens)):
            r0, r1 = int(query_start[b]), int(query_start[b + 1])
            L = int(context_lens[b])
            start = L - (r1 - r0)                      # position of the first new token
            for j in range(start // bs, -(-L // bs)) if r1 > r0 else ():
                blk = int(block_tables[b][j])
                a = max(start - j * bs, 0)             # earlier tokens fill slots 0 .. a-1
                e = min(L - j * bs, bs)
                rows = x[r0 + j * bs + a - start:r0 + j * bs + e - start]
                for h in range(H):
                    new = rows[:, h]
                    fin = np.abs(new[np.isfinite(new)])
                    old = float(scale[blk, h]) if a else 0.0
                    s = max(old, pow2_scale(fin.max() if fin.size else 0.0))
                    if a and s > old:
                        codes[blk, :a, h] = _encode_over(e4m3_decode(codes[blk, :a, h]) * old, s)
                    codes[blk, a:e, h] = _encode_over(new, s)
                    scale[blk, h] = s
    return tuple(outs)


def attention_weights(q, k_cache, block_tables, context_lens, scale):
    """Per sequence, the softmax weights summed over each KV head's query
    heads: a list of [Hkv, L_b] arrays."""
    q = _as_f64(q)
    Hkv = k_cache.shape[2]
    G = q.shape[1] // Hkv
    out = []
    for b in range(q.shape[0]):
        L = int(context_lens[b])
        K, _ = gather_context(k_cache, k_cache, block_tables[b], L)
        w = np.zeros((Hkv, L))
        for h in range(q.shape[1]) if L else ():
            s = (K[:, h // G] @ q[b, h]) * scale
            e = np.exp(s - s.max())
            w[h // G] += e / e.sum()
        out.append(w)
    return out


def evict(k_cache, v_cache, block_tables, context_lens, kept_lens, seen_lens, weights, token_pos, budget, recent,
          sinks, k_scale=None, v_scale=None):
    """Returns new (k_cache, v_cache, k_scale, v_scale, new_lens, weights, token_pos)."""
    kc, vc = np.array(k_cache, copy=True), np.array(v_cache, copy=True)
    ks = None if k_scale is None else np.array(k_scale, copy=True)
    vs = None if v_scale is None else np.array(v_scale, copy=True)
    bs, H = kc.shape[1], kc.shape[2]
    slots = block_tables.shape[1] * bs
    w_out, p_out = np.array(weights, copy=True), np.array(token_pos, copy=True)
    new_lens = np.array([min(int(L), budget) for L in context_lens], dtype=np.int32)
    for b, L in enumerate(int(x) for x in context_lens):
        new = min(L, budget)
        for h in range(H):
            pos = np.array([int(token_pos[b, h, t]) if t < kept_lens[b] else int(seen_lens[b]) - L + t
                            for t in range(L)], dtype=np.int64)
            safe = (pos < sinks) | (pos >= int(seen_lens[b]) - recent)
            w = np.array(weights[b, h, :L], dtype=np.float64)
            w[np.isnan(w)] = -np.inf
            order = sorted(range(L), key=lambda t: (not safe[t], -w[t] if not safe[t] else 0.0, t))
            kept = sorted(order[:new])
            stays, comes = [t for t in kept if t < new], [t for t in kept if t >= new]
            holes = [t for t in range(new) if t not in set(stays)]
            assert len(holes) == len(comes)
            source = dict(zip(stays, stays)) | dict(zip(holes, comes))
            w_out[b, h, :slots], p_out[b, h, :slots] = 0, -1
            for t, s in source.items():
                w_out[b, h, t], p_out[b, h, t] = weights[b, h, s], pos[s]
            if not holes:
                continue
            at = lambda t: (int(block_tables[b][t // bs]), t % bs, h)   # noqa: E731
            for old, pool, old_scale, sc in ((k_cache, kc, k_scale, ks), (v_cache, vc, v_scale, vs)):
                if sc is None:
                    for t, s in zip(holes, comes):
                        pool[at(t)] = old[at(s)]
                    continue
                for blk in sorted({at(t)[0] for t in holes}):
                    into = [(t, s) for t, s in zip(holes, comes) if at(t)[0] == blk]
                    was = float(old_scale[blk, h])
                    now = max([was] + [float(old_scale[at(s)[0], h]) for _, s in into])
                    if now > was:
                        for t in stays:
                            if at(t)[0] == blk:
                                pool[at(t)] = _encode_over(e4m3_decode(old[at(t)]) * was, now)
                    for t, s in into:
                        its = float(old_scale[at(s)[0], h])
                        pool[at(t)] = old[at(s)] if its == now else _encode_over(e4m3_decode(old[at(s)]) * its, now)
                    sc[blk, h] = now
    return kc, vc, ks, vs, new_lens, w_out, p_out
