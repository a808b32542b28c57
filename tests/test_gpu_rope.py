"""Rotary positions on the GPU against the oracle: layouts, partial heads, strides, far positions, in place, straight
into paged and latent caches, on another stream and in a captured graph.

Tolerance: the turn's fraction as a float is off by 2^-24 of at most a half turn (2^-22.3 of a radian), sincospif by
2^-22, the amplitude's product and the two multiplications by 2^-24 each: 2^-20 A (|x| + |y|) bounds their sum, and
the result is rounded once.  A step is off by 2^-65 of a turn and its frequency by 2^-51 of itself, on either side:
2^-50 |p| radians."""

import numpy as np
import pytest
import torch

import oracle
from _helpers import f64

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _check(got, x, pos, freq, amp, layout):
    x64 = f64(x)
    want = oracle.rope(x64, pos, freq, amp, layout)
    n = len(freq)
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    tol = HALF_STEP[x.dtype] * np.abs(want)
    size = amp * (np.abs(x64[..., a]) + np.abs(x64[..., b]))
    turn = 2.0 ** -20 + 2.0 ** -50 * np.abs(np.asarray(pos, dtype=np.float64))[:, None, None]
    tol[..., a] += size * turn
    tol[..., b] += size * turn
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), "worst %.3g of its bound" % (err / np.maximum(tol, 1e-300)).max()
    assert np.array_equal(f64(got)[..., 2 * n:], x64[..., 2 * n:])


POSITIONS = [0, 1, 2, 63, 4095, 131071, 1 << 20, (1 << 24) + 1, -1, -77, (1 << 31) - 1, -(1 << 31)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hkv,D,rot,kw", [
    (1, 1, 1, 16, 16, {}), (12, 5, 1, 32, 16, dict(scaling="linear", factor=8.0)), (33, 3, 2, 80, 48, {}),
    (7, 32, 8, 128, 128, dict(scaling="yarn", factor=32.0)), (700, 4, 4, 64, 32, dict(scaling="ntk", factor=4.0)),
    (2, 1, 0, 512, 512, {}), (401, 64, 8, 128, 64, {}), (5, 200, 9, 256, 80, {})])
def test_rope(pa, dtype, layout, N, Hq, Hkv, D, rot, kw):
    pos = (POSITIONS * (N // len(POSITIONS) + 1))[:N]
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    freq, amp = oracle.rope_frequencies(rot, 10000.0, **kw)
    steps, a = pa.rope_steps(rot, 10000.0, device="cuda", **kw)
    x = _randn(N, N, Hq + 2 * Hkv, D, dtype=dtype)
    q, k = x[:, :Hq], (x[:, Hq:Hq + Hkv] if Hkv else None)        # views into one projection's output
    q_out = torch.full((N, Hq, D), float("nan"), dtype=dtype, device="cuda")
    k_out = torch.full((N, Hkv, D), float("nan"), dtype=dtype, device="cuda") if Hkv else None
    before = x.clone()
    got = pa.rope(q, k, p, steps, amplitude=a, layout=layout, q_out=q_out, k_out=k_out)
    assert got[0] is q_out and got[1] is k_out and pa.last_error() == 0
    assert torch.equal(x, before)
    _check(q_out, q, pos, freq, amp, layout)
    if Hkv:
        _check(k_out, k, pos, freq, amp, layout)
    # in place: the same bits, the values' part untouched
    pa.rope(q, k, p, steps, amplitude=a, layout=layout)
    assert torch.equal(q, q_out) and (k is None or torch.equal(k, k_out))
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])


def test_rope_of_a_part_and_of_other_orders(pa):
    N, H = 37, 6
    pos = list(range(1000, 1000 + N))
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    freq, amp = oracle.rope_frequencies(64, 500000.0)
    steps, a = pa.rope_steps(64, 500000.0, device="cuda")
    x = _randn(3, N, H, 192)
    before = x.clone()
    pa.rope(x[:, :, 128:], None, p, steps, layout="interleaved")              # a head's last 64 elements
    assert torch.equal(x[:, :, :128], before[:, :, :128])
    _check(x[:, :, 128:], before[:, :, 128:], pos, freq, amp, "interleaved")
    y = _randn(4, H, N, 64).transpose(0, 1)                                   # heads outermost in memory
    out = torch.empty(H, N, 64, dtype=y.dtype, device="cuda").transpose(0, 1)
    pa.rope(None, y, p, steps, k_out=out)
    _check(out, y, pos, freq, amp, "half")
    one = _randn(5, N, 1, 64).expand(N, H, 64)                                # a broadcast input
    pa.rope(one, None, p, steps, q_out=out)
    _check(out, one, pos, freq, amp, "half")
    pa.rope(x[:0], None, p[:0], steps)                                        # no tokens
    assert pa.last_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hkv,D,rot,bs", [(1, 8, 8, 128, 128, 16), (50, 4, 1, 32, 16, 4), (300, 12, 4, 64, 32, 8),
                                               (19, 0, 3, 128, 64, 32)])
def test_rope_and_cache(pa, dtype, layout, N, Hq, Hkv, D, rot, bs):
    rng = np.random.default_rng(N)
    NB = N // bs + 3
    pos = rng.integers(0, 1 << 17, N).tolist()
    slots = rng.permutation(NB * bs)[:N].astype(np.int64)
    bad = N > 3
    if bad:
        slots[1], slots[2] = -5, NB * bs                          # padding, and a slot past the pool
    p, sl = torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.from_numpy(slots).cuda()
    freq, amp = oracle.rope_frequencies(rot, 10000.0, "yarn", 4.0)
    steps, a = pa.rope_steps(rot, 10000.0, scaling="yarn", factor=4.0, device="cuda")
    x = _randn(N + 1, N, Hq + 2 * Hkv, D, dtype=dtype)
    q, k, v = (x[:, :Hq] if Hq else None), x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    kc, vc = (_randn(i, NB, bs, Hkv, D, dtype=dtype) for i in (8, 9))
    k0, v0 = kc.clone(), vc.clone()
    q_out = torch.empty(N, Hq, D, dtype=dtype, device="cuda") if Hq else None
    pa.rope_and_cache(q, k, v, p, sl, kc, vc, steps, amplitude=a, layout=layout, q_out=q_out)
    assert pa.last_error() == (pa.DEV_BAD_SLOT if bad else 0)
    if Hq:
        _check(q_out, q, pos, freq, amp, layout)
    kept = [i for i in range(N) if 0 <= slots[i] < NB * bs]
    at = torch.from_numpy(slots[kept]).cuda()
    rows = lambda pool: pool.view(NB * bs, Hkv, D)               # noqa: E731
    _check(rows(kc)[at], k[kept], np.array(pos)[kept], freq, amp, layout)
    assert torch.equal(rows(vc)[at], v[kept])
    rest = torch.ones(NB * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(rows(kc)[rest], rows(k0)[rest]) and torch.equal(rows(vc)[rest], rows(v0)[rest])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,H,R,P,bs,layout", [(1, 128, 512, 64, 16, "interleaved"), (45, 3, 128, 16, 8, "half"),
                                               (900, 16, 384, 48, 32, "interleaved"), (64, 0, 256, 32, 16, "half")])
def test_latent_append(pa, dtype, N, H, R, P, bs, layout):
    rng = np.random.default_rng(N)
    NB = N // bs + 2
    pos = rng.integers(0, 1 << 16, N).tolist()
    slots = rng.permutation(NB * bs)[:N].astype(np.int64)
    bad = N > 3
    if bad:
        slots[0], slots[3] = -1, NB * bs + 7
    p, sl = torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.from_numpy(slots).cuda()
    freq, amp = oracle.rope_frequencies(P, 10000.0)
    steps, a = pa.rope_steps(P, 10000.0, device="cuda")
    down, q = _randn(1, N, R + P, dtype=dtype), _randn(2, N, max(H, 1), 128 + P, dtype=dtype)
    cache = _randn(3, NB, bs, R + P, dtype=dtype)
    before = cache.clone()
    qr = q[:, :, 128:] if H else None
    # into the rotary part of the absorbed queries
    absorbed = _randn(4, N, max(H, 1), R + P, dtype=dtype)
    q_out = absorbed[:, :, R:] if H else None
    pa.latent_append(down[:, :R], down[:, R:], p, sl, cache, steps, layout=layout, query=qr, query_out=q_out)
    assert pa.last_error() == (pa.DEV_BAD_SLOT if bad else 0)
    if H:
        _check(q_out, qr, pos, freq, amp, layout)
        assert torch.equal(absorbed[:, :, :R], _randn(4, N, H, R + P, dtype=dtype)[:, :, :R])
    kept = [i for i in range(N) if 0 <= slots[i] < NB * bs]
    at = torch.from_numpy(slots[kept]).cuda()
    rows = cache.view(NB * bs, R + P)
    assert torch.equal(rows[at, :R], down[kept, :R])
    _check(rows[at, R:][:, None], down[kept, R:][:, None], np.array(pos)[kept], freq, amp, layout)
    rest = torch.ones(NB * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(rows[rest], before.view(NB * bs, R + P)[rest])


def test_another_stream_and_a_captured_graph(pa):
    """A decode step's append captured, and replayed with other tokens, positions and slots in the same buffers."""
    N, H, Hkv, D, bs, NB = 9, 8, 2, 64, 16, 4
    steps, a = pa.rope_steps(D, device="cuda")
    p, sl = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int64, device="cuda")
    x = torch.zeros(N, H + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_out = torch.zeros(N, H, D, dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        pa.rope_and_cache(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], p, sl, kc, vc, steps, q_out=q_out, stream=stream)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    for seed in (1, 2, 3):
        x.copy_(_randn(seed, *x.shape))
        p.copy_(torch.arange(seed * 100, seed * 100 + N))
        sl.copy_(torch.randperm(NB * bs, device="cuda")[:N])
        kc.zero_(), vc.zero_()
        if seed < 3:
            g.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            step(side)
            torch.cuda.current_stream().wait_stream(side)
        freq, amp = oracle.rope_frequencies(D, 10000.0)
        pos = p.tolist()
        _check(q_out, x[:, :H], pos, freq, amp, "half")
        _check(kc.view(-1, Hkv, D)[sl], x[:, H:H + Hkv], pos, freq, amp, "half")
        assert torch.equal(vc.view(-1, Hkv, D)[sl], x[:, H + Hkv:])
    assert pa.last_error() == 0
