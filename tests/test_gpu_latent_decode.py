"""Attention over a paged latent cache (absorbed form) on the GPU against the oracle."""

import numpy as np
import pytest
import torch

from _latent import Cache, check, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _run(pa, c, q, scale, start=None, **kw):
    out = torch.full((*q.shape[:2], c.R), float("nan"), dtype=q.dtype, device="cuda")
    st = None if start is None else torch.tensor(start, dtype=torch.int32, device="cuda")
    got = pa.latent_decode(out, q, c.cache, c.table, c.lens, scale, query_start=st, **kw)
    assert got is out
    return out


@pytest.mark.parametrize("R,P", [(512, 64), (128, 16), (256, 32), (384, 48)])
@pytest.mark.parametrize("H,bs,lens", [(1, 16, [1]), (16, 16, [7, 130]), (128, 16, [300, 1, 128]), (5, 8, [127, 129, 640]),
                                       (32, 32, [33, 1000]), (64, 8, [256, 255]), (80, 16, [65, 2, 191]), (3, 32, [2100])])
def test_one_row_a_sequence(pa, R, P, H, bs, lens):
    c = Cache(lens, R, P, bs, seed=H)
    q = randn(H, len(lens), H, R + P)
    scale = 2.0 * (R + P) ** -0.5
    want = c.oracle(q, scale)
    check(_run(pa, c, q, scale), *want)
    assert pa.last_error() == 0


@pytest.mark.parametrize("R,P,H,bs,lens,new", [
    (512, 64, 16, 16, [40, 300, 5], [4, 1, 5]), (512, 64, 128, 16, [200, 131], [2, 3]), (256, 32, 3, 8, [64, 500, 20, 9], [30, 0, 20, 1]),
    (128, 64, 7, 32, [1000], [77]), (512, 64, 64, 16, [129, 128, 127], [1, 2, 1]), (384, 32, 1, 8, [300, 150], [150, 150])])
def test_several_rows_causal(pa, R, P, H, bs, lens, new):
    c = Cache(lens, R, P, bs, seed=len(lens))
    start = np.concatenate([[0], np.cumsum(new)])
    q = randn(R, int(start[-1]), H, R + P)
    scale = 2.0 * (R + P) ** -0.5
    want = c.oracle(q, scale, start)
    check(_run(pa, c, q, scale, start), *want)
    assert pa.last_error() == 0


def test_rows_with_nothing_to_see(pa):
    """A context of zero, more rows than context, rows behind the last sequence."""
    c = Cache([0, 3, 20], 512, 64, 16)
    start = [0, 2, 7, 8]                                  # sequence 1: five rows on three tokens
    q = randn(1, 11, 16, 576)
    want = c.oracle(q, 0.1, start)
    assert not want[0][:4].any()
    check(_run(pa, c, q, 0.1, start), *want)
    assert pa.last_error() == 0
    c = Cache([0, 40], 256, 32, 8)
    q = randn(1, 2, 4, 288)
    check(_run(pa, c, q, 0.1), *c.oracle(q, 0.1))


@pytest.mark.parametrize("H", [16, 128])
def test_scores_far_apart(pa, H):
    """One token takes nearly everything, early or late; scores that underflow beside it; growing maxima."""
    for seed, scale in ((1, 3.0), (2, 40.0)):
        c = Cache([700, 515], 512, 64, 16, seed=seed)
        q = randn(seed, 2, H, 576)
        check(_run(pa, c, q, scale * 576 ** -0.5), *c.oracle(q, scale * 576 ** -0.5))
    c = Cache([640], 128, 16, 16)
    for j in range(40):                                   # every block's keys larger than the last's
        c.cache[int(c.table[0, j])] *= 1.0 + j
    q = randn(5, 1, H, 144)
    check(_run(pa, c, q, 0.02), *c.oracle(q, 0.02))
    q = torch.zeros_like(q)                               # all scores equal
    check(_run(pa, c, q, 1.0), *c.oracle(q, 1.0))


def test_nan_stays_with_the_rows_that_see_it(pa):
    """A NaN in a key makes its rows NaN whole; later tokens' and other sequences' NaN do not show."""
    c = Cache([100, 60], 256, 32, 16)
    c.cache[int(c.table[0, 95 // 16]), 95 % 16, 280] = float("nan")     # the key part of token 95
    start = [0, 10, 12]
    q = randn(3, 12, 8, 288)
    out = _run(pa, c, q, 0.1, start)
    want = c.oracle(q, 0.1, start)
    assert torch.isnan(out[5:10]).all()                   # positions 95..99
    keep = [0, 1, 2, 3, 4, 10, 11]
    check(out[keep], *(x[keep] for x in want))


def test_nan_values_stay_with_the_rows_that_see_them(pa):
    """The same in the latent part, whose elements are the values too."""
    for H, R in ((8, 256), (16, 512)):
        c = Cache([100, 60], R, 32, 16)
        c.cache[int(c.table[0, 95 // 16]), 95 % 16, 70] = float("nan")
        start = [0, 10, 12]
        q = randn(3, 12, H, R + 32)
        out = _run(pa, c, q, 0.1, start)
        want = c.oracle(q, 0.1, start)
        assert torch.isnan(out[5:10]).all()
        keep = [0, 1, 2, 3, 4, 10, 11]
        check(out[keep], *(x[keep] for x in want))
    assert pa.last_error() == 0


@pytest.mark.parametrize("R,P", [(512, 64), (384, 16), (256, 48), (128, 32)])
@pytest.mark.parametrize("H,n,L", [(16, 1, 1500), (24, 1, 900), (64, 1, 1100), (128, 1, 700), (5, 3, 1000), (40, 4, 770)])
def test_many_tiles_a_cta(pa, R, P, H, n, L):
    """160 sequences over one context, whose maxima move in every tile: each is done by a CTA or two."""
    B = 160
    c = Cache([L], R, P, 16, seed=n)
    for j in range(-(-L // 16)):
        c.cache[int(c.table[0, j])] *= 1.0 + j / 16
    q = randn(H, n, H, R + P)
    scale = 0.5 * (R + P) ** -0.5
    want = c.oracle(q, scale, [0, n])
    c.table, c.lens = c.table.repeat(B, 1), c.lens.repeat(B)
    start = None if n == 1 else np.arange(B + 1) * n
    check(_run(pa, c, q.repeat(B, 1, 1), scale, start), *(np.tile(x, (B,) + (1,) * (x.ndim - 1)) for x in want))
    assert pa.last_error() == 0


@pytest.mark.parametrize("H", [16, 128])
def test_tokens_of_no_weight_before_low_scores(pa, H):
    """Scores of -inf in whole tiles at the start, then scores far below zero: as if the context began there."""
    B = 200                                               # (of one context: several tiles for every CTA)
    for L, hidden in ((300, 128), (700, 384), (150, 144)):
        c = Cache([L], 256, 32, 16, scale=0.5)
        q = randn(H, 1, H, 288)
        q[:, :, 280], q[:, :, 281] = 8.0, 1.0
        ids = c.table[0].long()
        c.cache[ids, :, 280] = -50.0                      # every score 400 lower
        c.cache[ids[:hidden // 16], :, 281] = -float("inf")
        rest = Cache([1], 256, 32, 16)
        rest.cache, rest.table, rest.lens = c.cache, c.table[:, hidden // 16:], c.lens - hidden
        want = rest.oracle(q, 1.0)
        c.table, c.lens = c.table.repeat(B, 1), c.lens.repeat(B)
        check(_run(pa, c, q.repeat(B, 1, 1), 1.0), *(x.repeat(B, 0) for x in want))
    assert pa.last_error() == 0


@pytest.mark.parametrize("H,lens", [(16, [20000]), (128, [9000, 30]), (40, [5000, 128, 0, 129, 7777])])
def test_long_sequences_cut_among_many(pa, H, lens):
    """Many CTAs a sequence, cuts at and inside tiles."""
    c = Cache(lens, 256, 32, 32, scale=0.5)
    q = randn(H, len(lens), H, 288)
    check(_run(pa, c, q, 0.2), *c.oracle(q, 0.2))
    assert pa.last_error() == 0


def test_bad_tables_and_lengths(pa):
    c = Cache([50, 90, 30], 512, 64, 16)
    q = randn(2, 3, 16, 576)
    want = c.oracle(q, 0.1)
    table = c.table.clone()
    c.table[1, 2] = 1 << 20                               # outside the pool: that sequence's own result only
    out = _run(pa, c, q, 0.1)
    assert pa.last_error() == pa.DEV_BAD_BLOCK
    check(out[[0, 2]], *(x[[0, 2]] for x in want))
    c.table.copy_(table)
    c.lens[0], c.lens[2] = -4, 30
    out = _run(pa, c, q, 0.1)
    assert pa.last_error() == pa.DEV_BAD_LEN and not out[0].any()
    check(out[1:], *(x[1:] for x in want))
    c.lens.copy_(torch.tensor([50, 90, 30]))
    # decreasing starts, and an end past the rows: those sequences write nothing
    for start, good in (([0, 2, 1, 3], [0, 2]), ([0, 1, 2, 9], [0, 1])):
        st = np.array(start)
        out = _run(pa, c, q, 0.1, start)
        assert pa.last_error() == pa.DEV_BAD_LEN
        for b in good:
            a, e = int(st[b]), int(st[b + 1])
            ref = c.oracle(q[a:e], 0.1, [0] * (b + 1) + [e - a] * (3 - b))
            mine = [i for i in range(e - a) if sum(st[s] <= a + i < st[s + 1] for s in good) == 1]   # (a row of two has no value)
            check(out[a:e][mine], *(x[mine] for x in ref))
    assert torch.isnan(out[2]).all()                      # the row of the sequence whose end lies past the rows


def test_long_context_and_offsets_past_32_bits(pa):
    """A pool of more than 2^32 bytes and elements, the sequence's blocks at its far end."""
    NB, bs, W = (1 << 32) // (16 * 576) + 200, 16, 576
    pool = torch.zeros(NB, bs, W, dtype=torch.bfloat16, device="cuda")
    L = 1500
    cols = -(-L // bs)
    ids = torch.randperm(190)[:cols] + NB - 190
    x = randn(7, cols * bs, W)
    pool[ids.cuda()] = x.view(cols, bs, W)
    c = Cache([1], 512, 64, bs)
    c.cache, c.table, c.lens = pool, ids.int().view(1, -1).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda")
    q = randn(8, 1, 16, W)
    out = _run(pa, c, q, 0.08)
    assert pa.last_error() == 0
    small = Cache([1], 512, 64, bs)
    small.cache, small.table, small.lens = x.view(cols, bs, W), torch.arange(cols, dtype=torch.int32, device="cuda")[None], c.lens
    check(out, *small.oracle(q, 0.08))
    assert torch.equal(out, _run(pa, small, q, 0.08))


def test_many_sequences(pa):
    lens = [(37 * i) % 200 + 1 for i in range(300)]
    c = Cache(lens, 128, 32, 16)
    q = randn(4, 300, 4, 160)
    check(_run(pa, c, q, 0.15), *c.oracle(q, 0.15))
    new = [i % 3 for i in range(300)]
    new = [min(n, L) for n, L in zip(new, lens)]
    start = np.concatenate([[0], np.cumsum(new)])
    q = randn(5, int(start[-1]), 4, 160)
    check(_run(pa, c, q, 0.15, start), *c.oracle(q, 0.15, start))
    assert pa.last_error() == 0


def test_same_bits_again_on_another_stream_and_in_graphs(pa):
    """Two captured graphs that share a workspace, replayed in turn with lengths that have grown in place."""
    c = Cache([900, 400], 512, 64, 16, cols=64)
    q = randn(1, 2, 128, 576)
    ws = pa.alloc_latent_workspace(q, c.cache, c.table)
    ws.fill_(0xFF)
    first = _run(pa, c, q, 0.08, workspace=ws)
    assert torch.equal(first, _run(pa, c, q, 0.08, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _run(pa, c, q, 0.08, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    q2 = randn(2, 2, 128, 576)
    outs = [torch.zeros(2, 128, 512, dtype=q.dtype, device="cuda") for _ in range(2)]
    graphs = []
    for out, x in zip(outs, (q, q2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.latent_decode(out, x, c.cache, c.table, c.lens, 0.08, workspace=ws)
        graphs.append(g)
    for lens in ([900, 400], [130, 77], [899, 1]):
        c.lens.copy_(torch.tensor(lens))
        for g in graphs:
            g.replay()
        for out, x in zip(outs, (q, q2)):
            assert torch.equal(out, _run(pa, c, x, 0.08, workspace=ws))
            check(out, *c.oracle(x, 0.08))
    assert pa.last_error() == 0


def test_two_calls_at_once(pa):
    """Calls on two streams, each with a workspace of its own."""
    c, d = Cache([700, 300, 5], 512, 64, 16, seed=1), Cache([2500], 256, 32, 8, seed=2)
    q, r = randn(1, 3, 40, 576), randn(2, 1, 16, 288)
    one, two = _run(pa, c, q, 0.08), _run(pa, d, r, 0.1)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, t):
        st.wait_stream(torch.cuda.current_stream())
    outs = [(_run(pa, c, q, 0.08, stream=s), _run(pa, d, r, 0.1, stream=t)) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, one) and torch.equal(y, two) for x, y in outs) and pa.last_error() == 0


def test_shared_blocks(pa):
    """Sequences whose tables share blocks, and one that names a block twice."""
    c = Cache([64, 64], 512, 64, 16, seed=3)
    c.table[1] = c.table[0]
    c.table[1, 2] = c.table[0, 1]
    q = randn(1, 2, 16, 576)
    check(_run(pa, c, q, 0.1), *c.oracle(q, 0.1))
    assert pa.last_error() == 0


def test_blocks_copied_and_swapped(pa):
    """Copy-on-write and swap of a latent pool's blocks: two layers a call, or one pool as both."""
    a, b = randn(1, 8, 16, 576), randn(2, 8, 16, 576)
    pairs = torch.tensor([[1, 5], [3, 0]], device="cuda")
    want_a, want_b = a.clone(), b.clone()
    for src, dst in pairs.tolist():
        want_a[dst], want_b[dst] = a[src], b[src]
    view = lambda x: x.view(8, 16, 1, 576)                 # noqa: E731
    pa.copy_blocks(view(a), view(b), pairs)
    assert torch.equal(a, want_a) and torch.equal(b, want_b)
    c, d = randn(3, 8, 16, 576), torch.zeros(8, 16, 576, dtype=torch.bfloat16, device="cuda")
    want = c.clone()
    want[5], want[0] = c[1], c[3]
    pa.copy_blocks(view(c), view(c), pairs)
    assert torch.equal(c, want)
    pa.swap_blocks(view(d), view(d), view(c), view(c), pairs)
    assert torch.equal(d[5], c[1]) and torch.equal(d[0], c[3]) and not d[1:5].any() and pa.last_error() == 0


def test_a_run_of_steps(pa):
    """Prompts appended, then tokens one step at a time: rotate and append, attend; the cache rebuilt by hand."""
    import oracle
    from _helpers import f64
    R, P, H, bs, B = 256, 32, 8, 16, 3
    lens = np.array([20, 1, 47])
    table = torch.randperm(16)[:B * 5].view(B, 5).int().cuda()
    cache = torch.zeros(16, bs, R + P, dtype=torch.bfloat16, device="cuda")
    steps, amp = pa.rope_steps(P, 10000.0, device="cuda")
    freq, _ = oracle.rope_frequencies(P, 10000.0)

    def slots(b, ts):
        return [int(table[b, t // bs]) * bs + t % bs for t in ts]

    for turn in range(4):
        new = lens if turn == 0 else np.ones(B, dtype=int)
        if turn:
            lens = lens + 1
        at = [t for b in range(B) for t in range(lens[b] - new[b], lens[b])]
        where = [s for b in range(B) for s in slots(b, range(lens[b] - new[b], lens[b]))]
        n = len(at)
        down, q = randn(turn, n, R + P), randn(10 + turn, n, H, 128 + P)
        full = torch.cat([randn(20 + turn, n, H, R), torch.zeros(n, H, P, dtype=q.dtype, device="cuda")], 2)
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        pa.latent_append(down[:, :R], down[:, R:], pos, torch.tensor(where, device="cuda"), cache, steps, layout="interleaved",
                         query=q[:, :, 128:], query_out=full[:, :, R:])
        turned = oracle.rope(f64(q[:, :, 128:]), at, freq, 1.0, "interleaved")
        assert np.abs(f64(full[:, :, R:]) - turned).max() <= np.abs(turned).max() * 2.0 ** -8 + 2.0 ** -18
        start = np.concatenate([[0], np.cumsum(new)])
        if turn == 0:
            # the prompts in the expanded form, their shared keys taken back from the cache
            up = randn(99, R, H * 256, scale=R ** -0.5)
            kv = (down[:, :R] @ up).view(n, H, 256)
            key = cache.view(-1, R + P)[torch.tensor(where, device="cuda")][:, R:]
            st = torch.tensor(start, dtype=torch.int32, device="cuda")
            got = pa.latent_prefill(torch.empty(n, H, 128, dtype=q.dtype, device="cuda"), q, st, kv, key, st, 0.08)
            check(got, *oracle.latent_prefill(f64(q), start, f64(kv), f64(key), start, 0.08))
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = torch.empty(n, H, R, dtype=q.dtype, device="cuda")
        pa.latent_decode(out, full, cache, table, ln, 0.1, query_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
        check(out, *oracle.latent_decode(f64(full), f64(cache), table.cpu().numpy(), lens.tolist(), 0.1, R, start))
    assert pa.last_error() == 0
