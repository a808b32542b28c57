"""Decode over the block-scaled e4m3 cache where one token takes nearly all the weight and its value is zero: the
output is then the sum of many tokens of small weight, and has to carry their digits."""

import numpy as np
import pytest
import torch

from _bounded import Case, check, u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _sink_case(Hq, Hkv, D, bs, L, share, at):
    """One sequence.  Token `at` has `share` of the weight of every head, and zeros as its value; the others'
    scores are spread around 0, and their values are positive."""
    c = Case("e4m3", [L], Hq, Hkv, D, bs, seed=L + D + Hq)
    G = Hq // Hkv
    for h in range(Hkv):
        c.q[0, h * G:(h + 1) * G] = c.q[0, h * G]
    c.ks[:] = 2.0 ** -8                              # scores with a deviation of 1/4
    c.vs[:] = 2.0 ** -6
    held = torch.from_numpy(c.used)
    c.v[held] &= 0x7F
    blk, i = int(c.tab[0, at // bs]), at % bs
    c.ks[blk] = 2.0 ** -4
    c.k[blk][held[blk]] = 0
    for h in range(Hkv):
        q = c.q[0, h * G].float()
        s = np.log(share / (1 - share) * L)
        k = q * (s / (float(q @ q) * c.scale))
        assert float(k.abs().max()) * 16 < 448
        c.k[blk, i, h] = (k * 16).to(torch.float8_e4m3fn).view(torch.uint8)
    c.v[blk, i] = 0
    return c


def _reference(c, share):
    """float64 outputs and the largest error an output may have.

    With p the softmax weights, A = sum p |v|, and w the largest weight:
      * the final rounding: u(bf16) |ref|;
      * each weight as terms of a narrow type: 2^-9 of itself, 2^-35 of the largest below their range,
        so 2^-9 A + L 2^-35 w max|v|;
      * a score is off by ds <= ((D + 4) 2^-24 + 2^-20) sum_d |q_d k_td| scale (fp32 products and sums, the query
        in terms of a narrower type), a weight by e^(2 ds);
      * 2^x, rescales and sums in fp32: (L + 64) 2^-23 relative."""
    K, V = c.f64_pools()
    L, G = int(c.lens[0]), c.Hq // c.Hkv
    blk = c.tab[0].long().numpy()[np.arange(L) // c.bs]
    K, V = K[blk, np.arange(L) % c.bs], V[blk, np.arange(L) % c.bs]
    q = c.q.double().numpy()
    ref, tol = np.zeros(c.q.shape), np.zeros(c.q.shape)
    for h in range(c.Hq):
        k, v = K[:, h // G], V[:, h // G]
        s = k @ q[0, h] * c.scale
        p = np.exp(s - s.max())
        p /= p.sum()
        top = p.max()
        assert (1 - share) / 2 < 1 - top < (1 - share) * 2     # (the sink's key is rounded to e4m3)
        ref[0, h] = p @ v
        A = p @ np.abs(v)
        ds = (np.abs(k * q[0, h]).sum(1) * c.scale).max() * ((c.D + 4) * 2.0 ** -24 + 2.0 ** -20)
        tol[0, h] = (u(torch.bfloat16) * np.abs(ref[0, h]) + L * 2.0 ** -35 * top * np.abs(v).max() +
                     (2.0 ** -9 + np.expm1(2 * ds) + (L + 64) * 2.0 ** -23) * A)
    return ref, tol


SHAPES = [(8, 2, 128, 16), (2, 2, 128, 16), (16, 2, 128, 8), (32, 2, 128, 32), (12, 2, 128, 16), (4, 4, 64, 16),
          (8, 2, 64, 16), (4, 4, 32, 16), (8, 8, 32, 8), (8, 2, 128, 4), (3, 3, 64, 16)]


@pytest.mark.parametrize("Hq,Hkv,D,bs", SHAPES)
@pytest.mark.parametrize("L,partition,share,at", [(2048, 0, 0.999, 0), (2048, -1, 0.9, 2047), (9000, -1, 0.999, 5),
                                                  (33000, 0, 0.999, 0), (33000, -1, 0.9999, 130)])
def test_decode_tail_beside_a_sink(pa, Hq, Hkv, D, bs, L, partition, share, at):
    c = _sink_case(Hq, Hkv, D, bs, L, share, at)
    ref, tol = _reference(c, share)
    c.cuda()
    out = torch.full_like(c.q, float("nan"))
    pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale, partition_size=partition)
    assert pa.last_error() == 0
    check(out, ref, tol)
    w = torch.zeros(1, Hkv, c.tab.shape[1] * bs, device="cuda")
    out.fill_(float("nan"))
    pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs,
                      partition_size=partition)
    assert pa.last_error() == 0
    check(out, ref, tol)
