"""Operators over an 8-bit paged KV cache with one scale per block and head, and of a cache of bounded
length: their workloads, their plain forms in elementary torch operations, and their definitions in 64 bits.

Operators
  append   new tokens quantised into an e4m3 pool, one power-of-two scale per (block, KV head)
  decode   one query per sequence over such a pool
  prefill  a chunk of each sequence's newest tokens, causal, over such a pool
  weights  decode that adds each token's softmax weight to a running total (f32, bf16 or e4m3 pools)
  evict    the cache of each (sequence, KV head) cut to a budget by those totals

Where ``own`` is false, ``run`` computes the plain form; where it is true it calls the package.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one new token per running request, many heads: the append of a decode step
        dict(name="append step 64 x 32 heads", op="append", B=64, Hkv=32, D=128, bs=16, src="bf16", ctx_min=128,
             ctx_max=2048, new_min=1, new_max=1),
        # prompts entering the cache in one call
        dict(name="append prompts 8 x 4096", op="append", B=8, Hkv=8, D=128, bs=16, src="bf16", ctx_min=4096,
             ctx_max=5120, new_min=3000, new_max=4096),
        # a few short requests with small heads: latency
        dict(name="decode 2 short", op="decode", B=2, Hq=8, Hkv=2, D=64, bs=8, ctx_min=1, ctx_max=300),
        # a batch of multi-head requests
        dict(name="decode 64 x 32 heads", op="decode", B=64, Hq=32, Hkv=32, D=128, bs=16, ctx_min=128, ctx_max=2048),
        # long contexts with grouped queries
        dict(name="decode 64 long grouped", op="decode", B=64, Hq=32, Hkv=8, D=128, bs=16, ctx_min=1024,
             ctx_max=16384),
        # a few requests with odd head groups in full precision: latency
        dict(name="weights 5 f32 odd groups", op="weights", B=5, Hq=12, Hkv=4, D=64, bs=4, pool="f32", ctx_min=1,
             ctx_max=700),
        # a bounded cache in 16 bits
        dict(name="weights 32 bf16 grouped", op="weights", B=32, Hq=32, Hkv=8, D=128, bs=16, pool="bf16",
             ctx_min=1024, ctx_max=8192),
        # the same in 8 bits, more requests
        dict(name="weights 64 e4m3 grouped", op="weights", B=64, Hq=32, Hkv=8, D=128, bs=16, pool="e4m3",
             ctx_min=1024, ctx_max=8192),
        # after a prompt: long contexts cut to a budget
        dict(name="evict 4 prompts", op="evict", B=4, Hkv=8, D=128, bs=16, pool="bf16", ctx_min=4096, ctx_max=16384,
             budget=2048, recent=256, sinks=4),
        # every step of a bounded cache: a few tokens over the budget, in 8 bits
        dict(name="evict step 64", op="evict", B=64, Hkv=8, D=128, bs=16, pool="e4m3", ctx_min=1025, ctx_max=1040,
             budget=1024, recent=128, sinks=4),
        # a mixed round: decode rows and short chunks together
        dict(name="prefill mixed 16", op="prefill", B=16, Hq=32, Hkv=8, D=128, bs=16, ctx_min=200, ctx_max=2048,
             new_min=1, new_max=100),
        # chunks of long prompts
        dict(name="prefill chunks 8 x 512", op="prefill", B=8, Hq=32, Hkv=8, D=128, bs=16, ctx_min=1024,
             ctx_max=4096, new_min=512, new_max=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "weights", "evict"])
    D = rng.choice([32, 64, 128, 128])
    bs = rng.choice([4, 8, 16, 16, 32])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
    B = _log(rng, 1, 64)
    if op == "append":
        ctx = _log(rng, 8, 4096)
        return dict(op=op, B=B, Hkv=Hkv, D=D, bs=bs, src=rng.choice(["bf16", "bf16", "f32"]),
                    ctx_min=max(1, ctx // 2), ctx_max=ctx, new_min=1,
                    new_max=max(1, min(ctx // 2, _log(rng, 1, 32768) // B)))
    G = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
    Hkv = min(Hkv, max(1, 64 // G))
    # up to half the largest listed decode's tokens x heads
    most = max(64, 300000 * 8 // (B * Hkv))
    ctx = _log(rng, 1, min(16384, most))
    lo = max(1, ctx // rng.choice([1, 2, 16]))
    if op == "decode":
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, ctx_min=lo, ctx_max=ctx)
    if op == "weights":
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, pool=rng.choice(["f32", "bf16", "e4m3", "e4m3"]),
                    ctx_min=min(lo, 4096), ctx_max=min(ctx, 8192))
    if op == "evict":
        budget = max(2, _log(rng, 8, 2048))
        recent = rng.randint(0, budget // 2)
        return dict(op=op, B=B, Hkv=Hkv, D=D, bs=bs, pool=rng.choice(["f32", "bf16", "e4m3", "e4m3"]),
                    ctx_min=max(1, min(budget, ctx) // 2), ctx_max=max(ctx, budget + rng.randint(1, 40)),
                    budget=budget, recent=recent, sinks=rng.randint(0, min(4, budget - recent)))
    G = rng.choice([1, 2, 4, 8, 16])
    Hkv = min(Hkv, max(1, 32 // G))
    B = min(B, 16)
    ctx = _log(rng, 4, 4096)
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=128, bs=rng.choice([8, 16, 32]), ctx_min=max(1, ctx // 2),
                ctx_max=ctx, new_min=1, new_max=max(1, min(ctx // 2, _log(rng, 1, 4096) // B)))


# --------------------------------------------------------------------- inputs

def _spread(lo, hi, n, gen):
    """n lengths evenly over lo..hi, in an order of the seed's: the sum, and with it every size, is the case's."""
    if n == 1:
        return torch.tensor([hi])
    x = lo + (hi - lo) * torch.arange(n) // (n - 1)
    return x[torch.randperm(n, generator=gen)]


def _gpu(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _scale_row(heads):
    """A scale row holds the heads rounded up to a multiple of four."""
    return (heads + 3) // 4 * 4


def _codes(shape, g):
    """e4m3 codes of N(0, 1) values over a scale of 2^-6, made a slice at a time."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - i),) + tuple(shape[1:]), generator=g, device="cuda") * 64.0
        out[i:i + step] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    return out


def _pool(c, kind, blocks, g):
    """K and V pools (and the scales of an e4m3 pool), as a serving program holds them."""
    shape = (blocks, c["bs"], c["Hkv"], c["D"])
    if kind != "e4m3":
        dt = torch.float32 if kind == "f32" else torch.bfloat16
        return dict(k=torch.randn(shape, generator=g, device="cuda").to(dt),
                    v=torch.randn(shape, generator=g, device="cuda").to(dt), k_scale=None, v_scale=None)
    sh = (blocks, _scale_row(c["Hkv"]))
    pow2 = [torch.exp2(torch.randint(-7, -4, sh, generator=g, device="cuda").float()) for _ in range(2)]
    return dict(k=_codes(shape, g), v=_codes(shape, g), k_scale=pow2[0], v_scale=pow2[1])


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    g = _gpu(seed)
    lens = _spread(c["ctx_min"], c["ctx_max"], c["B"], cpu)
    B, bs, Hkv, D = c["B"], c["bs"], c["Hkv"], c["D"]
    width = -(-c["ctx_max"] // bs)
    need = (lens + bs - 1) // bs
    blocks = int(need.sum()) + B
    order = torch.randperm(blocks, generator=cpu)
    first = torch.cumsum(need, 0) - need
    j = torch.arange(width)
    table = torch.where(j[None] < need[:, None], order[(first[:, None] + j[None]).clamp(max=blocks - 1)],
                        torch.tensor(blocks))
    s = dict(case=dict(c), lens=lens.int().cuda(), table=table.int().cuda(), max_len=int(lens.max()),
             scale=float(D) ** -0.5)
    kind = c.get("pool", "e4m3")
    s.update(_pool(c, kind, blocks, g))
    if c["op"] in ("append", "prefill"):
        n = _spread(c["new_min"], c["new_max"], B, cpu)
        start = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(n, 0)])
        s.update(start=start.int().cuda(), rows=int(start[-1]), max_new=int(n.max()))
    if c["op"] == "append":
        dt = torch.float32 if c["src"] == "f32" else torch.bfloat16
        s["key"] = torch.randn((s["rows"], Hkv, D), generator=g, device="cuda").to(dt)
        # values of very different size from head to head
        size = torch.exp2(torch.randint(-6, 7, (1, Hkv, 1), generator=g, device="cuda").float())
        s["value"] = (torch.randn((s["rows"], Hkv, D), generator=g, device="cuda") * size).to(dt)
    elif c["op"] == "evict":
        W = width * bs
        t = torch.arange(W, device="cuda")
        live = t[None, None] < s["lens"][:, None, None]
        # a few tokens hold most of the weight, and many hold none at all
        w = torch.randn((B, Hkv, W), generator=g, device="cuda").exp() ** 2
        w = torch.where(torch.rand((B, Hkv, W), generator=g, device="cuda") < 0.2, torch.zeros_like(w), w)
        s["weights"] = torch.where(live, w, torch.zeros_like(w))
        # half of the sequences have been cut before: their first tokens have positions of their own
        cut = torch.rand(B, generator=cpu) < 0.5
        kept = torch.where(cut, torch.minimum(lens, torch.tensor(c["budget"])), torch.zeros_like(lens))
        seen = torch.where(cut, lens + torch.randint(0, 5000, (B,), generator=cpu), lens)
        s["kept"], s["seen"] = kept.int().cuda(), seen.int().cuda()
        # ascending positions below seen - (L - kept), one of them for each kept token
        room = (seen - (lens - kept)).cuda()
        base = (torch.arange(W, device="cuda")[None] * room[:, None]) // kept.clamp(min=1).cuda()[:, None]
        s["pos"] = torch.where(t[None, None] < s["kept"][:, None, None], base[:, None].expand(B, Hkv, W),
                               torch.full((1,), -1, device="cuda")).int().contiguous()
        s["out"] = dict(new_lens=torch.empty_like(s["lens"]), weights=torch.empty_like(s["weights"]),
                        pos=torch.empty_like(s["pos"]))
    else:
        rows = s["rows"] if c["op"] == "prefill" else B
        dt = torch.float32 if kind == "f32" else torch.bfloat16
        s["q"] = torch.randn((rows, c["Hq"], D), generator=g, device="cuda").to(dt)
        s["out"] = torch.empty_like(s["q"])
        if c["op"] == "weights":
            s["weights"] = torch.rand((B, Hkv, width * bs), generator=g, device="cuda") * 4.0
            t = torch.arange(width * bs, device="cuda")
            s["weights"] *= t[None, None] < s["lens"][:, None, None]
    return s


def work(case):
    c = case
    B, Hkv, D, bs = c["B"], c["Hkv"], c["D"], c["bs"]
    L = (c["ctx_min"] + c["ctx_max"]) / 2.0
    elem = {"f32": 4, "bf16": 2, "e4m3": 1}[c.get("pool", "e4m3")]
    scales = 8.0 * Hkv / bs if elem == 1 else 0.0
    if c["op"] == "append":
        n = (c["new_min"] + c["new_max"]) / 2.0
        src = 4 if c["src"] == "f32" else 2
        return dict(bytes=B * n * 2 * Hkv * D * (src + 1) + B * (n / bs + 1) * 8 * Hkv, flops=B * n * 2 * Hkv * D)
    if c["op"] == "evict":
        slots = min(L, c["budget"])
        gone = max(0.0, L - c["budget"])
        # kept tokens fall on either side of the budget alike, but for the protected newest ones
        moved = gone * slots / max(L, 1.0)
        return dict(bytes=B * Hkv * (8.0 * L + 8.0 * slots + moved * 4 * D * elem), flops=B * Hkv * L)
    kv = B * L * (2.0 * Hkv * D * elem + scales)
    Hq = c["Hq"]
    if c["op"] == "prefill":
        n = (c["new_min"] + c["new_max"]) / 2.0
        return dict(bytes=kv + B * n * Hq * D * 4, flops=B * 4.0 * Hq * D * n * max(1.0, L - n / 2))
    qo = B * Hq * D * 2.0 * (4 if elem == 4 else 2)
    acc = B * L * 8.0 * Hkv if c["op"] == "weights" else 0.0
    return dict(bytes=kv + qo + acc, flops=4.0 * B * Hq * D * L)


# ----------------------------------------------------------------- plain forms

def _dequant(codes, scale, ids, Hkv):
    """Blocks ``ids`` of an e4m3 pool as fp32 values."""
    x = codes[ids].view(E4M3).float()
    return x * scale[ids][..., None, :Hkv, None]


def _context(s, which):
    """K or V of every sequence as fp32 [B, T, Hkv, D], zero past its length."""
    c = s["case"]
    cols = -(-s["max_len"] // c["bs"])
    t = torch.arange(cols * c["bs"], device="cuda")
    ids = s["table"][:, :cols].long()
    ids = torch.where(t[::c["bs"]][None] < s["lens"][:, None], ids, torch.zeros_like(ids))
    pool, scale = s[which], s[which + "_scale"]
    x = pool[ids].float() if scale is None else _dequant(pool, scale, ids, c["Hkv"])
    x = x.reshape(c["B"], cols * c["bs"], c["Hkv"], c["D"])
    live = t[None] < s["lens"][:, None]
    return torch.where(live[..., None, None], x, torch.zeros((), device="cuda")), live


def _softmax(x):
    """Over the last axis; a row with nothing in it gives zeros."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(s):
    c = s["case"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    K, live = _context(s, "k")
    q = s["q"].float().view(B, Hkv, -1, D)
    x = torch.matmul(q, K.permute(0, 2, 3, 1)) * s["scale"]
    del K
    x = torch.where(live[:, None, None], x, torch.full((), -math.inf, device="cuda"))
    p = _softmax(x)
    V, _ = _context(s, "v")
    out = torch.matmul(p, V.permute(0, 2, 1, 3)).reshape(B, -1, D).to(s["q"].dtype)
    return out, p


def _plain_weights(s):
    out, p = _plain_decode(s)
    n = p.shape[-1]
    s["weights"][..., :n] += p.sum(2)
    return dict(out=out, weights=s["weights"])


def _plain_prefill(s):
    c = s["case"]
    B, Hkv, D, N = c["B"], c["Hkv"], c["D"], s["max_new"]
    start, lens = s["start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(N, device="cuda")
    row = (start[:-1, None] + i[None]).clamp(max=s["rows"] - 1)
    G = c["Hq"] // Hkv
    q = s["q"][row].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    K, _ = _context(s, "k")
    x = torch.matmul(q, K.permute(0, 2, 3, 1)).view(B, Hkv, N, G, -1) * s["scale"]
    t = torch.arange(x.shape[-1], device="cuda")
    see = t[None, None] <= (lens - n)[:, None, None] + i[None, :, None]
    x = torch.where(see[:, None, :, None], x, torch.full((), -math.inf, device="cuda"))
    V, _ = _context(s, "v")
    o = torch.matmul(_softmax(x).view(B, Hkv, N * G, -1), V.permute(0, 2, 1, 3))
    o = o.view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D)
    return o[i[None] < n[:, None]].to(s["q"].dtype)


def _pow2_scale(a):
    """The smallest power of two s with a <= 448 s, at least MIN_SCALE; 0 for 0."""
    m, e = torch.frexp(a)
    s = torch.ldexp(torch.ones_like(a), torch.where(m <= 0.875, e - 9, e - 8))
    return torch.where(a > 0, s.clamp(min=MIN_SCALE), torch.zeros_like(a))


def _encode(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)


def _plain_append_one(s, which, src):
    c = s["case"]
    bs, Hkv = c["bs"], c["Hkv"]
    start, lens = s["start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    lo = (lens - n) // bs
    j = lo[:, None] + torch.arange(s["max_new"] // bs + 2, device="cuda")[None]
    b, u = torch.nonzero((j * bs < lens[:, None]) & (n[:, None] > 0), as_tuple=True)
    blk = s["table"][b, j[b, u]].long()
    pos = j[b, u][:, None] * bs + torch.arange(bs, device="cuda")[None]
    old = pos < (lens - n)[b][:, None]
    new = ~old & (pos < lens[b][:, None])
    row = (start[:-1][b][:, None] + pos - (lens - n)[b][:, None]).clamp(0, s["rows"] - 1)
    x = torch.where(new[..., None, None], src[row].float(), torch.zeros((), device="cuda"))
    pool, scale = s[which], s[which + "_scale"]
    was = torch.where(old[:, :1], scale[blk][:, :Hkv], torch.zeros((), device="cuda"))
    now = torch.maximum(was, _pow2_scale(x.abs().amax((1, 3))))
    by = torch.where(now > 0, now, torch.ones_like(now))[:, None, :, None]
    fresh = _encode(x / by)
    kept = _encode(pool[blk].view(E4M3).float() * (was[:, None, :, None] / by))
    code = torch.where(new[..., None, None], fresh, torch.where(old[..., None, None], kept, pool[blk]))
    pool[blk] = code
    scale[blk, :Hkv] = now


def _plain_append(s):
    _plain_append_one(s, "k", s["key"])
    _plain_append_one(s, "v", s["value"])
    return _pool_out(s)


def _pool_out(s):
    """The pools as the values that their codes stand for, and the scales."""
    if s["k_scale"] is None:
        return dict(k=s["k"], v=s["v"])
    return dict(k=s["k"].view(E4M3), v=s["v"].view(E4M3), k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_evict(s):
    c = s["case"]
    B, Hkv, bs, W = c["B"], c["Hkv"], c["bs"], s["weights"].shape[2]
    lens, kept, seen = (s[n].long()[:, None, None] for n in ("lens", "kept", "seen"))
    t = torch.arange(W, device="cuda")[None, None]
    live = t < lens
    pos = torch.where(t < kept, s["pos"].long(), seen - lens + t)
    safe = (pos < c["sinks"]) | (pos >= seen - c["recent"])
    key = torch.where(safe, torch.full((), math.inf, device="cuda"), s["weights"])
    key = torch.where(live, key, torch.full((), -math.inf, device="cuda"))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    stay = torch.zeros((B, Hkv, W), dtype=torch.bool, device="cuda").scatter_(
        2, order[..., :c["budget"]], torch.ones((), dtype=torch.bool, device="cuda").expand(B, Hkv, min(W, c["budget"])))
    stay &= live
    hole = ~stay & (t < torch.clamp(lens, max=c["budget"]))
    come = stay & (t >= c["budget"])
    b, h, dst = torch.nonzero(hole, as_tuple=True)
    _, _, src = torch.nonzero(come, as_tuple=True)           # as many in every (b, h), in the same order
    new_len = torch.clamp(lens, max=c["budget"])
    w = torch.where(stay & (t < new_len), s["weights"], torch.zeros((), device="cuda"))
    p = torch.where(stay & (t < new_len), pos, torch.full((), -1, device="cuda"))
    w[b, h, dst] = s["weights"][b, h, src]
    p[b, h, dst] = pos[b, h, src]
    table = s["table"].long()
    db, sb = table[b, dst // bs], table[b, src // bs]
    if c["pool"] != "e4m3":
        for pool in (s["k"], s["v"]):
            pool[db, dst % bs, h] = pool[sb, src % bs, h]
    else:
        for pool, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            was = scale.clone()
            up = torch.zeros_like(scale).view(-1).scatter_reduce_(
                0, db * scale.shape[1] + h, was[sb, h], "amax").view_as(scale)
            scale.copy_(torch.maximum(was, up))
            # the rows that stay in a block whose scale has grown
            grown = up > was
            bb, hh, tt = torch.nonzero(stay & (t < new_len), as_tuple=True)
            rb = table[bb, tt // bs]
            pick = grown[rb, hh]
            rb, hh, tt = rb[pick], hh[pick], tt[pick] % bs
            moved = pool[sb, src % bs, h].view(E4M3).float() * (was[sb, h] / _or_one(scale[db, h]))[:, None]
            pool[rb, tt, hh] = _encode(pool[rb, tt, hh].view(E4M3).float() * (was[rb, hh] / scale[rb, hh])[:, None])
            pool[db, dst % bs, h] = _encode(moved)
    return dict(_pool_out(s), weights=w, pos=p.int(), new_lens=new_len.view(-1).int())


def _or_one(x):
    return torch.where(x > 0, x, torch.ones_like(x))


# -------------------------------------------------------------------------- run

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    if op == "append":
        return _plain_append(s)
    if op == "decode":
        return _plain_decode(s)[0]
    if op == "prefill":
        return _plain_prefill(s)
    if op == "weights":
        return _plain_weights(s)
    return _plain_evict(s)


def _own(s, op):
    from paged_kv_cache_307_gb300 import _lib as pa
    c = s["case"]
    cache = (s["k"], s["v"])
    scales = (s["k_scale"], s["v_scale"])
    where = (s["table"], s["lens"])
    if op == "append":
        pa.append_fp8_blocks(s["key"], s["value"], s["start"], *where, *cache, *scales)
        return _pool_out(s)
    if op == "prefill":
        return pa.prefill_fp8_blocks(s["out"], s["q"], s["start"], *cache, *scales, *where, s["scale"])
    if "workspace" not in s:         # a serving program keeps it from step to step
        s["workspace"] = (pa.alloc_evict_workspace(s["k"], s["table"], c["budget"]) if op == "evict" else
                          pa.alloc_weights_workspace(s["q"], s["k"], s["table"]) if op == "weights" else
                          pa.alloc_fp8_blocks_workspace(s["q"], s["k"], s["table"]))
    ws = s["workspace"]
    if op == "decode":
        return pa.decode_fp8_blocks(s["out"], s["q"], *cache, *scales, *where, s["scale"], workspace=ws)
    if op == "weights":
        pa.decode_weights(s["out"], s["weights"], s["q"], *cache, *where, s["scale"], k_scale=scales[0],
                          v_scale=scales[1], workspace=ws)
        return dict(out=s["out"], weights=s["weights"])
    o = s["out"]
    pa.evict(*cache, *where, s["kept"], s["seen"], s["weights"], s["pos"], c["budget"], o["new_lens"], o["weights"],
             o["pos"], recent=c["recent"], sinks=c["sinks"], k_scale=scales[0], v_scale=scales[1], workspace=ws)
    return dict(_pool_out(s), weights=o["weights"], pos=o["pos"], new_lens=o["new_lens"])


# ------------------------------------------------- the definitions, in 64 bits

def _f64_value(codes):
    """e4m3 codes as float64, from the format: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    c = torch.arange(256, dtype=torch.float64)
    e, m = torch.floor(c / 8) % 16, c % 8
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
    v[127] = math.nan
    v[128:] = -v[:128]
    return v.cuda()[codes.long()]


def _f64_round(x):
    """x to the nearest e4m3 value (ties to the even mantissa), at most 448 in size."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > x.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _f64_rows(s, which, b, L):
    """The first L rows of sequence b, [L, Hkv, D] in float64."""
    c = s["case"]
    ids = s["table"][b, :-(-L // c["bs"])].long()
    x = s[which][ids]
    if s[which + "_scale"] is None:
        x = x.double()
    else:
        x = _f64_value(x) * s[which + "_scale"][ids][:, None, :c["Hkv"], None].double()
    return x.reshape(-1, c["Hkv"], c["D"])[:L]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(s)
    if op == "evict":
        return _exact_evict(s)
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    lens = s["lens"].tolist()
    start = s["start"].tolist() if op == "prefill" else list(range(c["B"] + 1))
    outs = []
    totals = s["weights"].double() if op == "weights" else None
    for b, L in enumerate(lens):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        K, V = _f64_rows(s, "k", b, L), _f64_rows(s, "v", b, L)
        q = s["q"][start[b]:start[b + 1]].double().view(n, c["Hkv"], G, c["D"])
        o = torch.empty_like(q)
        for h in range(c["Hkv"]):
            x = q[:, h].reshape(n * G, -1) @ K[:, h].T * s["scale"]
            at = torch.arange(L - n, L, device="cuda").repeat_interleave(G)
            x[torch.arange(L, device="cuda")[None] > at[:, None]] = -math.inf
            p = torch.softmax(x, -1)
            o[:, h] = (p @ V[:, h]).view(n, G, -1)
            if totals is not None:
                totals[b, h, :L] += p.sum(0)
        outs.append(o.view(n, c["Hq"], c["D"]))
    out = torch.cat(outs)
    return dict(out=out, weights=totals) if op == "weights" else out


def _exact_append(s):
    c = s["case"]
    bs, Hkv = c["bs"], c["Hkv"]
    start, lens, table = s["start"].tolist(), s["lens"].tolist(), s["table"].tolist()
    got = {}
    for which, src in (("k", s["key"]), ("v", s["value"])):
        value = _f64_value(s[which])
        scale = s[which + "_scale"].double()
        # a group of equal spans at a time: (first slot, last slot) of the new tokens within a block
        spans = {}
        for b, L in enumerate(lens):
            n = start[b + 1] - start[b]
            p = L - n
            while p < L:
                end = min(L, (p // bs + 1) * bs)
                spans.setdefault((p % bs, end - p), []).append((table[b][p // bs], start[b] + p - (L - n)))
                p = end
        for (a, n), found in spans.items():
            blk = torch.tensor([f[0] for f in found], device="cuda")
            row = torch.tensor([f[1] for f in found], device="cuda")[:, None] + torch.arange(n, device="cuda")
            x = src[row].double()
            top = x.abs().amax((1, 3))
            need = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
            # a logarithm just above a whole number
            need = torch.where(top <= need / 2 * E4M3_MAX, need / 2, need).clamp(min=MIN_SCALE)
            need = torch.where(top > 0, need, torch.zeros_like(top))
            before = scale[blk, :Hkv] if a else torch.zeros_like(need)
            after = torch.maximum(before, need)
            div = torch.where(after > 0, after, torch.ones_like(after))[:, None, :, None]
            if a:
                value[blk, :a] = _f64_round(value[blk, :a] * before[:, None, :, None] / div)
            value[blk, a:a + n] = _f64_round(x / div)
            scale[blk, :Hkv] = after
        got[which], got[which + "_scale"] = value, scale
    return got


def _exact_evict(s):
    c = s["case"]
    bs, budget = c["bs"], c["budget"]
    table = s["table"].long()
    q = c["pool"] == "e4m3"
    pools = {w: _f64_value(s[w]) if q else s[w].double() for w in ("k", "v")}
    scales = {w: s[w + "_scale"].double() for w in ("k", "v")} if q else None
    before = {w: scales[w].clone() for w in ("k", "v")} if q else None
    W = s["weights"].shape[2]
    weights = torch.zeros((c["B"], c["Hkv"], W), dtype=torch.float64)
    lens, kept, seen = s["lens"].tolist(), s["kept"].tolist(), s["seen"].tolist()
    w_all, p_all = s["weights"].double().cpu(), s["pos"].cpu()
    pos_out = torch.full((c["B"], c["Hkv"], W), -1, dtype=torch.int32)
    for b, L in enumerate(lens):
        t = torch.arange(L)
        new = min(L, budget)
        for h in range(c["Hkv"]):
            pos = torch.where(t < kept[b], p_all[b, h, :L].long(), seen[b] - L + t)
            w = w_all[b, h, :L]
            rank = torch.where((pos < c["sinks"]) | (pos >= seen[b] - c["recent"]), torch.full_like(w, math.inf), w)
            chosen = torch.sort(rank, descending=True, stable=True).indices[:new].sort().values
            stays, comes = chosen[chosen < new], chosen[chosen >= new]
            free = torch.ones(new, dtype=torch.bool)
            free[stays] = False
            holes = torch.nonzero(free).view(-1)
            place = torch.cat([stays, holes])
            source = torch.cat([stays, comes])
            weights[b, h, place] = w[source]
            pos_out[b, h, place] = pos[source].int()
            if not len(holes):
                continue
            holes, comes, stays = holes.cuda(), comes.cuda(), stays.cuda()
            db, sb, rb = table[b, holes // bs], table[b, comes // bs], table[b, stays // bs]
            for name in ("k", "v"):
                x, at = pools[name], (db, holes % bs, h)
                if not q:
                    x[at] = x[sb, comes % bs, h]
                    continue
                sc, was = scales[name], before[name]
                grown = was[:, h].clone()
                grown.scatter_reduce_(0, db, was[sb, h], "amax")
                sc[table[b, :-(-new // bs)], h] = grown[table[b, :-(-new // bs)]]
                one = torch.ones((), dtype=torch.float64, device="cuda")
                rows = _f64_round(x[rb, stays % bs, h] * (was[rb, h] / torch.where(sc[rb, h] > 0, sc[rb, h], one))[:, None])
                x[rb, stays % bs, h] = torch.where((sc[rb, h] > was[rb, h])[:, None], rows, x[rb, stays % bs, h])
                x[at] = _f64_round(x[sb, comes % bs, h] * (was[sb, h] / torch.where(sc[db, h] > 0, sc[db, h], one))[:, None])
    got = dict(k=pools["k"], v=pools["v"], weights=weights.cuda(), pos=None, new_lens=None)
    if q:
        got.update(k_scale=scales["k"], v_scale=scales["v"])
    return got
