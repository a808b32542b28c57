"""Cases and derived tolerances shared by the tests of the block-scaled e4m3
cache, the weight-keeping decode and the eviction.

Tolerances.  u(t) = finfo(t).eps / 2 is the most a rounding to type t is off,
relative to the value.  For one output element, with p the softmax weights and
A = sum p |v|:
  * the final rounding: u(out) |ref|;
  * softmax weights rounded to at least 8 significant bits before the product
    with V on the tensor-core paths (bf16, f16, or two e4m3 terms): 2^-8 A, and
    below the normal range of the rounded type an absolute 2^-22 of the largest
    weight for each token: L 2^-22 max|v|.  CUDA cores and f32 pools: none;
  * a score is off by ds <= (D + 4) 2^-24 max_t sum_d |q_d k_td| scale (a chain of
    D fp32 products and sums, the prescaled query, the scale), and 2^-20 of the
    largest |q k| sum where the query is split into terms of a narrower type;
    a weight then by a factor e^(2 ds), the normaliser's shift included;
  * 2^x, the running rescales and the sum over L tokens in fp32:
    (L + 64) 2^-23 relative.
"""

import numpy as np
import torch

import oracle


def u(t):
    return float(torch.finfo(t).eps) / 2


class Case:
    """Random pools, tables and lengths, the slots no sequence holds filled with NaN (codes)."""

    def __init__(self, pool, lens, Hq, Hkv, D, bs, seed=0, spare_cols=2, codes_nan=True, rows=None):
        rng = np.random.default_rng(seed)
        self.pool, self.Hq, self.Hkv, self.D, self.bs = pool, Hq, Hkv, D, bs
        lens = np.asarray(lens, dtype=np.int32)
        B = len(lens)
        need = -(-lens // bs)
        NB = int(need.sum()) + 3
        order = rng.permutation(NB)
        width = int(max(1, need.max())) + spare_cols
        tab = np.full((B, width), NB + 7, dtype=np.int32)      # unused entries name no block
        used = np.zeros((NB, bs), dtype=bool)
        o = 0
        for b in range(B):
            tab[b, :need[b]] = order[o:o + need[b]]
            for j in range(need[b]):
                used[tab[b, j], :min(bs, lens[b] - j * bs)] = True
            o += need[b]
        self.used = used
        g = torch.Generator().manual_seed(seed)
        shape = (NB, bs, Hkv, D)
        if pool == "e4m3":
            def codes():
                c = (torch.randn(shape, generator=g) * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                c[~torch.from_numpy(used)] = 0x7F if codes_nan else 0
                return c
            self.k, self.v = codes(), codes()
            row = (Hkv + 3) // 4 * 4
            s = [torch.exp2(torch.from_numpy(rng.integers(-7, -4, (NB, row)).astype(np.float32))) for _ in range(2)]
            self.ks, self.vs = s
            self.qt = torch.bfloat16
        else:
            self.qt = torch.float32 if pool == "f32" else torch.bfloat16
            self.k = torch.randn(shape, generator=g).to(self.qt)
            self.v = torch.randn(shape, generator=g).to(self.qt)
            self.k[~torch.from_numpy(used)] = float("nan")
            self.v[~torch.from_numpy(used)] = float("nan")
            self.ks = self.vs = None
        self.q = torch.randn((B if rows is None else rows, Hq, D), generator=g).to(self.qt)
        self.tab, self.lens = torch.from_numpy(tab), torch.from_numpy(lens)
        self.scale = float(np.float32(1 / np.sqrt(D)))

    def cuda(self):
        for n in ("k", "v", "ks", "vs", "q", "tab", "lens"):
            t = getattr(self, n)
            if t is not None:
                setattr(self, n, t.cuda())
        return self

    def f64_pools(self):
        """The pools in float64, slots no sequence holds as zeros."""
        k, v = (x.cpu() for x in (self.k, self.v))
        if self.pool == "e4m3":
            out = [oracle.dequantize_blocks(x.numpy(), s.cpu().numpy()) for x, s in ((k, self.ks), (v, self.vs))]
        else:
            out = [x.double().numpy() for x in (k, v)]
        return [np.where(self.used[:, :, None, None], x, 0.0) for x in out]


def reference(c, query_start=None):
    """float64 outputs and the largest error an output may have."""
    K, V = c.f64_pools()
    q, tab, lens = c.q.cpu().double().numpy(), c.tab.cpu().numpy(), c.lens.cpu().numpy()
    tab = np.where(tab < K.shape[0], tab, 0)
    if query_start is None:
        att = lambda v: oracle.paged_decode(q, K, v, tab, lens, c.scale)      # noqa: E731
    else:
        att = lambda v: oracle.paged_prefill_varlen(q, query_start, K, v, tab, lens, c.scale)   # noqa: E731
    ref, A = att(V), att(np.abs(V))
    L = max(1, int(lens.max()))
    narrow = 0.0 if c.pool == "f32" else 1.0
    ds = score_error(c, q, K)
    tol = (u(c.qt) * np.abs(ref) + narrow * (2 ** -8 * A + L * 2.0 ** -22 * np.abs(V).max()) +
           (np.expm1(2 * ds) + (L + 64) * 2.0 ** -23) * A + 1e-30)
    return ref, tol


def score_error(c, q, K):
    G = c.Hq // c.Hkv
    most = 0.0
    for h in range(c.Hkv):
        k = np.abs(K[:, :, h]).reshape(-1, c.D)
        most = max(most, float((np.abs(q[:, h * G:(h + 1) * G]).reshape(-1, c.D) @ k.T).max()))
    return most * c.scale * ((c.D + 4) * 2.0 ** -24 + (2.0 ** -20 if c.pool == "e4m3" else 0.0))


def check(got, ref, tol):
    got = got.detach().cpu().double().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - ref) / tol
    assert off.max() <= 1, "off by %.3g times the tolerance at %s" % (off.max(), np.unravel_index(off.argmax(), off.shape))
