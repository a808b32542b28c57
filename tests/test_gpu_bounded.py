"""A cache of bounded length through the C ABI against the oracle: decode that keeps the weights, eviction,
and the steps of a request together (eager and as a captured graph)."""

import numpy as np
import pytest
import torch

import oracle
from _bounded import Case, check, reference, score_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


# ------------------------------------------------------------------ decode with weights

LENS = [1, 0, 15, 16, 17, 300, 700, 129, 256]


def _totals(c, start):
    """The oracle's totals from `start`, and the tolerance: relative to a weight e^(2 ds), 2^x and the sums
    (L + 64) 2^-23 and G additions; the addition to the total half a step of it."""
    K, _ = c.f64_pools()
    tab = np.where(c.tab.cpu().numpy() < K.shape[0], c.tab.cpu().numpy(), 0)
    q = c.q.cpu().double().numpy()
    w = oracle.attention_weights(q, K, tab, c.lens.cpu().numpy(), c.scale)
    ref = start.double().numpy().copy()
    tol = np.full(ref.shape, 1e-30)
    L = max(1, int(c.lens.max()))
    rel = np.expm1(2 * score_error(c, q, K)) + (L + 64 + c.Hq // c.Hkv) * 2.0 ** -23
    for b, x in enumerate(w):
        ref[b, :, :x.shape[1]] += x
        # (weights below the range of normal fp32 numbers may vanish)
        tol[b, :, :x.shape[1]] += rel * x + 2.0 ** -24 * ref[b, :, :x.shape[1]] + 2.0 ** -120
    return ref, tol


@pytest.mark.parametrize("pool,Hq,Hkv,D,bs", [
    ("f32", 4, 4, 32, 4), ("f32", 12, 4, 64, 8), ("f32", 8, 2, 128, 16), ("bf16", 8, 8, 128, 16), ("bf16", 8, 2, 128, 16),
    ("bf16", 16, 2, 64, 8), ("bf16", 6, 2, 64, 32), ("bf16", 16, 1, 128, 16), ("bf16", 32, 1, 128, 16),
    ("bf16", 32, 8, 128, 16), ("e4m3", 8, 8, 128, 16), ("e4m3", 32, 8, 128, 16), ("e4m3", 14, 2, 128, 32),
    ("e4m3", 4, 2, 64, 8), ("e4m3", 3, 3, 32, 4), ("e4m3", 32, 2, 128, 16), ("e4m3", 6, 3, 128, 8), ("e4m3", 5, 1, 128, 16)])
@pytest.mark.parametrize("partition", [0, 64])
def test_weights(pa, pool, Hq, Hkv, D, bs, partition):
    c = Case(pool, LENS, Hq, Hkv, D, bs, seed=Hq + bs)
    ref, tol = reference(c)
    g = torch.Generator().manual_seed(1)
    slots = c.tab.shape[1] * bs + 3                          # rows longer than the table
    start = torch.rand(len(LENS), Hkv, slots, generator=g)
    wref, wtol = _totals(c, start)
    c.cuda()
    out, w = torch.full_like(c.q, float("nan")), start.cuda()
    pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs,
                      partition_size=partition)
    assert pa.last_error() == 0
    check(out, ref, tol)
    check(w, wref, wtol)
    for b, L in enumerate(LENS):                             # nothing past the context is touched
        assert torch.equal(w[b, :, L:].cpu(), start[b, :, L:])
    # the same call gives the same bits
    again, w2 = torch.empty_like(out), start.cuda()
    pa.decode_weights(again, w2, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs,
                      partition_size=partition)
    assert torch.equal(w, w2)
    assert torch.equal(again, out)


def test_weights_sharp_softmax(pa):
    """A token that takes all the weight, scores far below the range of 2^x."""
    for pool in ("f32", "bf16", "e4m3"):
        c = Case(pool, [400, 33], 8, 2, 128, 16, seed=2)
        c.q *= 40.0
        ref, tol = reference(c)
        start = torch.zeros(2, 2, c.tab.shape[1] * 16)
        wref, wtol = _totals(c, start)
        c.cuda()
        out, w = torch.empty_like(c.q), start.cuda()
        pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs)
        assert pa.last_error() == 0
        check(out, ref, tol)
        check(w, wref, wtol)


@pytest.mark.parametrize("pool,Hq,Hkv,D", [("f32", 4, 2, 32), ("bf16", 4, 4, 128), ("bf16", 8, 2, 128), ("e4m3", 4, 4, 64)])
def test_weights_nan_key_makes_nan_of_its_head(pa, pool, Hq, Hkv, D):
    c = Case(pool, [150, 1], Hq, Hkv, D, 16, seed=6)
    c.k[c.tab[0, 1].long(), 3, 1, 5] = 0x7F if pool == "e4m3" else float("nan")
    c.k[c.tab[1, 0].long(), 0, 0, 5] = 0x7F if pool == "e4m3" else float("nan")
    c.cuda()
    out, w = torch.empty_like(c.q), torch.zeros(2, Hkv, c.tab.shape[1] * 16, device="cuda")
    pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, k_scale=c.ks, v_scale=c.vs)
    assert pa.last_error() == 0
    G = Hq // Hkv
    nan = torch.zeros(out.shape, dtype=torch.bool)
    nan[0, G:2 * G] = True
    nan[1, :G] = True
    assert torch.equal(out.isnan().cpu(), nan)
    wn = torch.zeros(w.shape, dtype=torch.bool)
    wn[0, 1, :150] = True
    wn[1, 0, :1] = True
    assert torch.equal(w.isnan().cpu(), wn)


def test_weights_many_sequences(pa):
    rng = np.random.default_rng(0)
    c = Case("bf16", rng.integers(0, 40, 1100), 4, 2, 64, 16, seed=1)
    start = torch.zeros(1100, 2, c.tab.shape[1] * 16)
    wref, wtol = _totals(c, start)
    ref, tol = reference(c)
    c.cuda()
    out, w = torch.empty_like(c.q), start.cuda()
    pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale)
    assert pa.last_error() == 0
    check(out, ref, tol)
    check(w, wref, wtol)


# ------------------------------------------------------------------ eviction

def _evict_inputs(pool, lens, Hkv, D, bs, budget, seed=0, kept=(), ties=False, extra=0):
    c = Case(pool, lens, Hkv, Hkv, D, bs, seed=seed, spare_cols=1, codes_nan=False)
    if pool != "e4m3":
        c.k, c.v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    rng = np.random.default_rng(seed)
    B, slots = len(lens), c.tab.shape[1] * bs + extra
    w = rng.integers(0, 3, (B, Hkv, slots)) if ties else rng.standard_normal((B, Hkv, slots)) ** 2
    w = torch.from_numpy(w.astype(np.float32))
    seen = np.array(lens, dtype=np.int32)
    kl = np.zeros(B, dtype=np.int32)
    pos = np.full((B, Hkv, slots), -1, dtype=np.int32)
    for b in kept:
        kl[b] = min(lens[b], budget)
        seen[b] = lens[b] + 1000
        for h in range(Hkv):
            pos[b, h, :kl[b]] = rng.permutation(int(seen[b]) - (lens[b] - kl[b]))[:kl[b]]
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x))      # noqa: E731
    return c, w, t(pos), t(kl), t(seen)


def _evict_both(pa, c, w, pos, kl, seen, budget, recent, sinks, in_place):
    n = lambda x: None if x is None else x.numpy()               # noqa: E731
    bits = lambda x: x.view(torch.int16).numpy() if x.dtype == torch.bfloat16 else x.numpy()   # noqa: E731
    ref = oracle.evict(bits(c.k), bits(c.v), c.tab.numpy(), c.lens.numpy(), kl.numpy(), seen.numpy(), w.numpy(),
                       pos.numpy(), budget, recent, sinks, n(c.ks), n(c.vs))
    c.cuda()
    w, pos, kl, seen = w.cuda(), pos.cuda(), kl.cuda(), seen.cuda()
    slots = c.tab.shape[1] * c.bs
    if in_place:
        wo, po, new = w, pos, c.lens
    else:
        wo, po, new = torch.full_like(w, 5.0), torch.full_like(pos, 5), torch.empty_like(c.lens)
    pa.evict(c.k, c.v, c.tab, c.lens, kl, seen, w, pos, budget, new, wo, po, recent=recent, sinks=sinks, k_scale=c.ks,
             v_scale=c.vs)
    code = pa.last_error()
    k2, v2, ks2, vs2, new2, w2, p2 = ref
    assert np.array_equal(new.cpu().numpy(), new2)
    assert np.array_equal(wo.cpu().numpy()[..., :slots], w2[..., :slots])
    assert np.array_equal(po.cpu().numpy()[..., :slots], p2[..., :slots])
    if not in_place:
        assert (wo[..., slots:] == 5).all() and (po[..., slots:] == 5).all()
    assert np.array_equal(bits(c.k.cpu()), k2) and np.array_equal(bits(c.v.cpu()), v2)
    if ks2 is not None:
        assert np.array_equal(c.ks.cpu().numpy(), ks2) and np.array_equal(c.vs.cpu().numpy(), vs2)
    return code


@pytest.mark.parametrize("pool", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,D,bs,budget,recent,sinks", [(2, 128, 16, 64, 16, 4), (3, 32, 4, 37, 0, 0), (1, 64, 8, 1, 1, 0),
                                                          (2, 64, 32, 100, 100, 0), (8, 128, 16, 129, 7, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(pa, pool, Hkv, D, bs, budget, recent, sinks, in_place):
    lens = [0, 1, budget, budget + 1, 2 * budget + 3, 700, budget - 1, 513, 2 * budget]
    args = _evict_inputs(pool, lens, Hkv, D, bs, budget, seed=budget, kept=(2, 4, 5), extra=5)
    assert _evict_both(pa, *args, budget, recent, sinks, in_place) == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_evict_ties_go_to_the_lower_slot(pa, pool):
    args = _evict_inputs(pool, [1500, 600, 90], 2, 64, 16, 80, ties=True)
    assert _evict_both(pa, *args, 80, 10, 2, True) == 0


def test_evict_all_equal_negative_and_not_finite_weights(pa):
    c, w, pos, kl, seen = _evict_inputs("bf16", [300, 300, 300, 300], 2, 64, 16, 100)
    w[0] = 0.0
    w[1] = -w[1]
    w[2, :, ::3], w[2, :, 1::7] = float("inf"), float("nan")
    w[3, :, ::2], w[3, :, 1::2] = -0.0, 0.0
    assert _evict_both(pa, c, w, pos, kl, seen, 100, 0, 0, False) == 0


@pytest.mark.parametrize("L", [4097, 70001, 200003])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_context(pa, L, in_place):
    args = _evict_inputs("bf16", [L, 5, 2500], 1, 32, 32, 2048, seed=5, ties=L < 5000)
    assert _evict_both(pa, *args, 2048, 256, 4, in_place) == 0


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens", [[2100, 2049, 300], [5000] * 2 + [1200] * 38])
def test_evict_long_rows_few_and_many(pa, lens, ties):
    """Six and eighty rows of more than 2048 slots: another split of the selection each."""
    args = _evict_inputs("e4m3", lens, 2, 32, 32, 1024, seed=6, ties=ties)
    assert _evict_both(pa, *args, 1024, 64, 4, ties) == 0


def test_evict_lengths_out_of_range_are_clamped_and_flagged(pa):
    c, w, pos, kl, seen = _evict_inputs("bf16", [40, 40], 2, 64, 16, 16)
    c.lens[0] = -3
    kl[1] = 99
    pos[1] = torch.arange(pos.shape[2]).int()
    n = c.tab.shape[1] * 16
    k, v = c.k.clone(), c.v.clone()
    c.cuda()
    new, wo, po = torch.empty_like(c.lens), torch.empty_like(w).cuda(), torch.empty_like(pos).cuda()
    pa.evict(c.k, c.v, c.tab, c.lens, kl.cuda(), seen.cuda(), w.cuda(), pos.cuda(), 16, new, wo, po)
    assert pa.last_error() == pa.DEV_BAD_LEN
    assert new.tolist() == [0, 16]
    assert (wo[0, :, :n] == 0).all() and (po[0, :, :n] == -1).all()
    b = c.tab[0, :3].long().cpu()
    assert torch.equal(c.k.cpu()[b].view(torch.int16), k[b].view(torch.int16))


def test_evict_moves_from_and_to_bad_blocks_are_skipped(pa):
    c, w, pos, kl, seen = _evict_inputs("bf16", [64], 1, 64, 16, 32)
    w[:] = 0
    w[0, 0, 40], w[0, 0, 60] = 5.0, 6.0              # slots 30 and 31 are freed
    c.tab[0, 3] = 10 ** 6                            # the block of slot 60
    k = c.k.clone()
    t = c.tab.clone()
    c.cuda()
    new, wo, po = torch.empty_like(c.lens), torch.empty_like(w).cuda(), torch.empty_like(pos).cuda()
    pa.evict(c.k, c.v, c.tab, c.lens, kl.cuda(), seen.cuda(), w.cuda(), pos.cuda(), 32, new, wo, po)
    assert pa.last_error() == pa.DEV_BAD_BLOCK
    k[t[0, 1].long(), 14] = k[t[0, 2].long(), 8]
    assert torch.equal(c.k.cpu(), k)
    assert po[0, 0, 30:32].tolist() == [40, 60]


# ------------------------------------------------------------------ a request's steps together

class _Loop:
    """Append, weight-keeping decode and eviction over one small batch, every buffer fixed (so that a step can
    be captured), and the same with the oracle."""

    def __init__(self, pa, pool, B=3, Hq=8, Hkv=2, D=128, bs=16, budget=40, over=3):
        self.pa, self.pool, self.budget, self.over = pa, pool, budget, over
        self.B, self.Hq, self.Hkv, self.D, self.bs = B, Hq, Hkv, D, bs
        cols = -(-(budget + over) // bs)
        NB = B * cols + 1
        g = torch.Generator().manual_seed(11)
        self.tab = torch.randperm(NB, generator=g)[:B * cols].int().view(B, cols).cuda()
        if pool == "e4m3":
            self.k, self.v = (torch.zeros(NB, bs, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.ks, self.vs = (torch.zeros(NB, 4, device="cuda") for _ in range(2))
        else:
            self.k, self.v = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.ks = self.vs = None
        i = dict(dtype=torch.int32, device="cuda")
        self.lens, self.kept, self.seen = (torch.zeros(B, **i) for _ in range(3))
        self.w = torch.zeros(B, Hkv, cols * bs, device="cuda")
        self.pos = torch.full((B, Hkv, cols * bs), -1, **i)
        self.q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        self.key, self.val = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.out = torch.zeros_like(self.q)
        self.start = torch.arange(B + 1, **i)
        self.scale = D ** -0.5
        self.ws = pa.alloc_weights_workspace(self.q, self.k, self.tab)
        self.wse = pa.alloc_evict_workspace(self.k, self.tab, budget)
        self.gen = torch.Generator(device="cuda").manual_seed(5)

    def feed(self):
        for x in (self.q, self.key, self.val):
            x.copy_(torch.randn(x.shape, generator=self.gen, device="cuda"))

    def step(self):
        pa = self.pa
        self.lens += 1
        self.seen += 1
        if self.pool == "e4m3":
            pa.append_fp8_blocks(self.key, self.val, self.start, self.tab, self.lens, self.k, self.v, self.ks, self.vs)
        else:
            t = self.lens.long() - 1
            slots = self.tab.gather(1, (t // self.bs)[:, None]).view(-1).long() * self.bs + t % self.bs
            pa.reshape_and_cache(self.key, self.val, slots, self.k, self.v)
        pa.decode_weights(self.out, self.w, self.q, self.k, self.v, self.tab, self.lens, self.scale, k_scale=self.ks,
                          v_scale=self.vs, workspace=self.ws)

    def cut(self):
        self.pa.evict(self.k, self.v, self.tab, self.lens, self.kept, self.seen, self.w, self.pos, self.budget,
                      self.lens, self.w, self.pos, recent=8, sinks=2, k_scale=self.ks, v_scale=self.vs,
                      workspace=self.wse)
        self.kept.copy_(self.lens)

    def state(self):
        return [x.clone() for x in (self.out, self.w, self.pos, self.lens, self.k, self.v) +
                ((self.ks, self.vs) if self.ks is not None else ())]


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_steps_of_a_bounded_cache_against_plain_attention(pa, pool):
    """70 steps under a budget of 40: the kept tokens' rows, positions and totals stay together, and attention
    over the cut cache is attention over those tokens."""
    L = _Loop(pa, pool)
    rows = []                                       # every token's key and value as the cache holds it
    for i in range(70):
        L.feed()
        rows.append((L.key.double().cpu().numpy(), L.val.double().cpu().numpy()))
        before = L.w.clone()
        L.step()
        n = int(L.lens[0])
        assert n == min(i + 1, 40 + (0 if i < 40 else (i - 40) % 3 + 1))
        grown = (L.w - before).sum(-1)
        # 40 fp32 weights and totals, each off by at most 2^-22 of a sum below 2^9
        assert torch.allclose(grown, torch.full_like(grown, 4.0), atol=1e-3)
        if n == 43:
            L.cut()
            for h in range(2):
                p = L.pos[0, h, :40].cpu().numpy()
                assert len(set(p.tolist())) == 40 and {0, 1} <= set(p.tolist())
                assert set(range(i + 1 - 8, i + 1)) <= set(p.tolist())
    assert pa.last_error() == 0
    # the cache holds the rows of the positions it says it holds
    for b in range(L.B):
        n, kept, seen = int(L.lens[b]), int(L.kept[b]), int(L.seen[b])
        for h in range(2):
            pos = [int(L.pos[b, h, t]) if t < kept else seen - n + t for t in range(n)]
            for x, sc, which in ((L.k, L.ks, 0), (L.v, L.vs, 1)):
                got = x.cpu()[L.tab[b].long().cpu()]
                if pool == "e4m3":
                    got = oracle.dequantize_blocks(got.numpy(), sc.cpu().numpy()[L.tab[b].long().cpu().numpy()])
                    scale = np.repeat(sc.cpu().numpy()[L.tab[b].long().cpu().numpy()][:, h], L.bs)[:n, None]
                    got = got.reshape(-1, 2, 128)[:n, h]
                    want = np.stack([rows[p][which][b, h] for p in pos])
                    # one rounding to e4m3 (2^-4) and, under a raised scale, half a subnormal step a raise
                    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 4 * 2.0 ** -10 * scale).all()
                else:
                    got = got.double().numpy().reshape(-1, 2, 128)[:n, h]
                    assert np.array_equal(got, np.stack([rows[p][which][b, h] for p in pos]))


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_captured_steps_give_the_eager_bits(pa, pool):
    def run(graph):
        L = _Loop(pa, pool)
        if graph:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                L.step()
                L.cut()
            torch.cuda.current_stream().wait_stream(s)
            for x in (L.lens, L.seen, L.kept, L.w, L.k, L.v) + ((L.ks, L.vs) if L.ks is not None else ()):
                x.zero_()
            L.pos.fill_(-1)
            gs, gc = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(gs):
                L.step()
            with torch.cuda.graph(gc):
                L.cut()
        for i in range(50):
            L.feed()
            gs.replay() if graph else L.step()
            if i >= 42 and i % 2 == 0:
                gc.replay() if graph else L.cut()
        torch.cuda.synchronize()
        assert pa.last_error() == 0
        return L.state()
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_two_streams_two_workspaces(pa):
    """Two batches on two streams at once, each with its own workspace, give what they give alone."""
    a, b = _Loop(pa, "bf16"), _Loop(pa, "e4m3")
    def run(L):
        for i in range(45):
            L.feed()
            L.step()
            if i == 42:
                L.cut()
    run(a)
    run(b)
    torch.cuda.synchronize()
    want = a.state(), b.state()
    a, b = _Loop(pa, "bf16"), _Loop(pa, "e4m3")
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(45):
        for L, s in ((a, sa), (b, sb)):
            with torch.cuda.stream(s):
                L.feed()
                L.step()
                if i == 42:
                    L.cut()
    torch.cuda.synchronize()
    for L, w in ((a, want[0]), (b, want[1])):
        assert all(torch.equal(x, y) for x, y in zip(L.state(), w))
    assert pa.last_error() == 0


@pytest.mark.parametrize("pool", ["f32", "bf16", "e4m3"])
def test_empty_contexts_in_a_long_table(pa, pool):
    """Nothing to look at: zeros come out and the running totals stay, whatever the partitions."""
    c = Case(pool, [0, 0, 0], 8, 2, 128, 16, spare_cols=400).cuda()
    w = torch.full((3, 2, c.tab.shape[1] * 16), 3.0, device="cuda")
    for partition in (0, 64, -1):
        out = torch.full_like(c.q, float("nan"))
        sc = dict(k_scale=c.ks, v_scale=c.vs) if pool == "e4m3" else {}
        pa.decode_weights(out, w, c.q, c.k, c.v, c.tab, c.lens, c.scale, partition_size=partition, **sc)
        assert (out == 0).all() and (w == 3.0).all()
    assert pa.last_error() == 0
