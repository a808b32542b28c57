"""Inputs and bounds shared by the GPU tests of latent attention.

Bound of an output element: the softmax weights are rounded to bf16 (2^-8 of each, so 2^-8 of sum w |v|), the output
is rounded once (2^-8 of itself), and a score is a sum of at most 576 fp32 products: off by less than 2^-18 of
scale max_t sum |q k|, which moves every weight by that much of itself, on both sides of the quotient.  (2^x and the
fp32 sums add 2^-18.)"""

import numpy as np
import torch

import oracle
from _helpers import f64


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def check(got, want, mass, size):
    """want may be NaN: rows of no sequence, which got holds NaN for as well."""
    got = f64(got)
    free = np.isnan(want)
    assert np.isnan(got[free]).all(), "rows of no sequence were written"
    tol = 2.0 ** -8 * (mass + np.abs(want)) + (2.0 ** -17 * size[..., None] + 2.0 ** -17) * mass
    err = np.abs(got - want)
    bad = ~(err <= tol) & ~free
    assert not bad.any(), "%d of %d off, worst %.3g of its bound, first %s" % (
        bad.sum(), bad.size, np.nanmax(err / np.maximum(tol, 1e-300)), np.argwhere(bad)[0])


class Cache:
    """A latent cache with one table row a sequence, garbage (NaN) everywhere that no sequence owns."""

    def __init__(self, lens, R, P, bs, seed=0, cols=None, scale=1.0):
        rng = np.random.default_rng(seed)
        need = [-(-L // bs) for L in lens]
        NB = sum(need) + 3
        ids = rng.permutation(NB)
        cols = cols or max(1, max(need))
        table = np.full((len(lens), cols), NB + 5, dtype=np.int32)      # entries past the context are not ids
        pool = torch.full((NB, bs, R + P), float("nan"), dtype=torch.bfloat16, device="cuda")
        at = 0
        for b, L in enumerate(lens):
            table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            x = randn(seed * 1000 + b, L, R + P, scale=scale)
            for j in range(need[b]):
                n = min(bs, L - j * bs)
                pool[int(table[b, j]), :n] = x[j * bs:j * bs + n]
        self.cache, self.R, self.P, self.bs = pool, R, P, bs
        self.table, self.lens = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def oracle(self, q, scale, start=None, lens=None):
        lens = self.lens.tolist() if lens is None else lens
        return oracle.latent_decode(f64(q), f64(self.cache), self.table.cpu().numpy(), lens, scale, self.R, start)
