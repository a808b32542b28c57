"""Rotary positions and attention over a cache of one latent vector a token: their workloads, their plain forms
in elementary torch operations, and their definitions in 64 bits.

Operators
  rope           queries and keys rotated by their positions
  rope_cache     the same, the keys (and the values beside them) straight into a paged cache
  latent_append  a token's latent vector and its rotated shared key into a paged latent cache, the rotary part of
                 its queries rotated along
  latent_decode  attention of each sequence's newest tokens over a latent cache, in the absorbed form: a query
                 meets the latent vectors themselves, and they are the values
  latent_prefill ragged causal attention in the expanded form: keys and values of every head, one rotated key
                 shared by all heads

Where ``own`` is false, ``run`` computes the plain form; where it is true it calls the package.
"""

import math

import torch

own = False

BASE = 10000.0
YARN = dict(factor=32.0, original=4096.0, beta_fast=32.0, beta_slow=1.0)


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of a few requests: latency
        dict(name="rope step 4", op="rope", N=4, Hq=32, Hkv=8, D=128, rot=128, layout="half", scaling="none", far=4096,
             src="bf16"),
        # a prompt's worth of tokens, context stretched 32 times
        dict(name="rope prompt 8192", op="rope", N=8192, Hq=32, Hkv=8, D=128, rot=128, layout="interleaved",
             scaling="yarn", far=131072, src="bf16"),
        # the append of a decode step, many heads
        dict(name="rope append step 64", op="rope_cache", N=64, Hq=32, Hkv=32, D=128, rot=128, layout="half",
             scaling="none", far=2048, src="bf16", bs=16),
        # prompts in full precision, half of each head rotated
        dict(name="rope append prompts f32", op="rope_cache", N=5000, Hq=12, Hkv=4, D=64, rot=32, layout="half",
             scaling="linear", far=16384, src="f32", bs=4),
        # a decode step over a latent cache: 64 requests' new tokens, the queries of 128 heads
        dict(name="latent append step 64", op="latent_append", N=64, H=128, R=512, P=64, layout="interleaved",
             scaling="yarn", far=65536, src="bf16", bs=16),
        # prompts entering a latent cache, 16 heads on this GPU
        dict(name="latent append prompts 16384", op="latent_append", N=16384, H=16, R=512, P=64, layout="interleaved",
             scaling="yarn", far=65536, src="bf16", bs=16),
        # two short requests, few heads: latency
        dict(name="latent decode 2 short", op="latent_decode", B=2, H=16, R=512, P=64, bs=16, ctx_min=1, ctx_max=300,
             new_min=1, new_max=1, src="bf16"),
        # long contexts, the heads divided among GPUs
        dict(name="latent decode 64 long x 16 heads", op="latent_decode", B=64, H=16, R=512, P=64, bs=16, ctx_min=1024,
             ctx_max=16384, new_min=1, new_max=1, src="bf16"),
        # the whole model's heads on one GPU
        dict(name="latent decode 64 x 128 heads", op="latent_decode", B=64, H=128, R=512, P=64, bs=16, ctx_min=1024,
             ctx_max=8192, new_min=1, new_max=1, src="bf16"),
        # drafted tokens checked in one pass, a smaller latent vector, an odd batch
        dict(name="latent decode 11 drafts", op="latent_decode", B=11, H=32, R=256, P=32, bs=8, ctx_min=300,
             ctx_max=5000, new_min=1, new_max=5, src="bf16"),
        # a mixed round of short chunks behind contexts of their own
        dict(name="latent prefill mixed 7", op="latent_prefill", B=7, H=8, Dn=128, P=64, Dv=128, ctx_min=340,
             ctx_max=1500, new_min=1, new_max=333, src="bf16"),
        # whole prompts
        dict(name="latent prefill 4 x 4096", op="latent_prefill", B=4, H=32, Dn=128, P=64, Dv=128, ctx_min=4096,
             ctx_max=4096, new_min=4096, new_max=4096, src="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_cache", "latent_append", "latent_decode", "latent_decode", "latent_prefill",
                     "latent_prefill"])
    turn = dict(layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                far=_log(rng, 64, 1 << 20), src=rng.choice(["bf16", "bf16", "f32"]))
    bs = rng.choice([4, 8, 16, 16, 32])
    if op in ("rope", "rope_cache"):
        D = rng.choice([32, 64, 128, 128])
        Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 8])
        N = max(1, min(_log(rng, 1, 8192), 8192 * 40 * 128 // ((Hq + 2 * Hkv) * D)))
        c = dict(op=op, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([16, D // 2, D, D]), **turn)
        return dict(c, bs=bs) if op == "rope_cache" else c
    H = rng.choice([1, 3, 8, 16, 16, 32, 64, 128])
    if op == "latent_append":
        return dict(op=op, N=max(1, min(_log(rng, 1, 16384), 16384 * 16 // H)), H=H, R=rng.choice([128, 256, 384, 512, 512]),
                    P=rng.choice([32, 64, 64]), bs=max(8, bs), **turn)
    B = _log(rng, 1, 64)
    if op == "latent_decode":
        new = rng.choice([1, 1, 1, 2, 4, 7])
        # up to half the largest listed case's tokens x heads
        ctx = max(new, _log(rng, 1, max(64, min(16384, 64 * 4608 * 64 // (B * H * new)))))
        return dict(op=op, B=B, H=H, R=rng.choice([128, 256, 384, 512, 512, 512]), P=rng.choice([32, 64, 64]),
                    bs=rng.choice([8, 16, 16, 32]), ctx_min=max(new, ctx // rng.choice([1, 2, 16])), ctx_max=ctx,
                    new_min=1, new_max=new, src="bf16")
    B, H = min(B, 16), rng.choice([1, 3, 8, 16, 32])
    ctx = _log(rng, 2, 4096)
    new = max(1, min(ctx // rng.choice([1, 1, 2, 8]), 4 * 4096 * 4096 * 32 // (B * H * ctx)))
    Dn, P, Dv = rng.choice([(128, 64, 128), (128, 64, 128), (64, 32, 64), (128, 32, 64)])
    return dict(op=op, B=B, H=H, Dn=Dn, P=P, Dv=Dv, ctx_min=max(new, ctx // rng.choice([1, 2])), ctx_max=ctx,
                new_min=max(1, new // rng.choice([1, 4])), new_max=new, src="bf16")


# --------------------------------------------------------------------- inputs

def _spread(lo, hi, n, gen):
    """n lengths evenly over lo..hi, in an order of the seed's: the sum, and with it every size, is the case's."""
    if n == 1:
        return torch.tensor([hi])
    x = lo + (hi - lo) * torch.arange(n) // (n - 1)
    return x[torch.randperm(n, generator=gen)]


def _starts(n):
    return torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(n, 0)])


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if c["src"] == "f32" else torch.bfloat16

    def randn(*shape):
        return torch.randn(shape, generator=gpu, device="cuda", dtype=dt)

    s = dict(case=dict(c))
    if c["op"] in ("rope", "rope_cache", "latent_append"):
        N = c["N"]
        # runs of consecutive positions, as the chunks of a batch have them
        first = torch.randint(0, c["far"], (N,), generator=cpu)
        run = torch.arange(N) % 64
        s["pos"] = ((first[torch.arange(N) - run] + run) % c["far"]).int().cuda()
        if c["op"] != "rope":
            bs = c["bs"]
            blocks = -(-N // bs) + 8
            slots = torch.randperm(blocks, generator=cpu)[:, None] * bs + torch.arange(bs)
            s["slots"] = slots.reshape(-1)[:N].cuda()
        if c["op"] == "latent_append":
            # the down-projection's output holds the latent vector and the shared key side by side, a head of the
            # queries its two parts
            down, q = randn(N, c["R"] + c["P"]), randn(N, c["H"], 128 + c["P"])
            s.update(latent=down[:, :c["R"]], key=down[:, c["R"]:], q=q[:, :, 128:],
                     cache=torch.zeros(blocks, bs, c["R"] + c["P"], dtype=dt, device="cuda"),
                     q_out=torch.empty(N, c["H"], c["P"], dtype=dt, device="cuda"))
        else:
            # one projection's output: queries, keys and values side by side
            Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
            x = randn(N, Hq + 2 * Hkv, D)
            s.update(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:],
                     q_out=torch.empty(N, Hq, D, dtype=dt, device="cuda"))
            if c["op"] == "rope":
                s["k_out"] = torch.empty(N, Hkv, D, dtype=dt, device="cuda")
            else:
                s["k_cache"], s["v_cache"] = (torch.zeros(blocks, bs, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
        return s
    B, H = c["B"], c["H"]
    lens = _spread(c["ctx_min"], c["ctx_max"], B, cpu)
    new = torch.minimum(_spread(c["new_min"], c["new_max"], B, cpu), lens)
    start = _starts(new)
    rows = int(start[-1])
    s.update(lens=lens.int().cuda(), start=start.int().cuda(), rows=rows, max_len=int(lens.max()),
             max_new=int(new.max()))
    if c["op"] == "latent_decode":
        R, P, bs = c["R"], c["P"], c["bs"]
        width = -(-c["ctx_max"] // bs)
        need = (lens + bs - 1) // bs
        blocks = int(need.sum()) + B
        order = torch.randperm(blocks, generator=cpu)
        first = torch.cumsum(need, 0) - need
        j = torch.arange(width)
        table = torch.where(j[None] < need[:, None], order[(first[:, None] + j[None]).clamp(max=blocks - 1)],
                            torch.tensor(blocks))
        s.update(table=table.int().cuda(), cache=randn(blocks, bs, R + P), q=randn(rows, H, R + P),
                 out=torch.empty(rows, H, R, dtype=dt, device="cuda"),
                 # scores of standard deviation two: a few tokens hold most of the weight
                 scale=2.0 * float(R + P) ** -0.5)
        return s
    kv_start = _starts(lens)
    total = int(kv_start[-1])
    s.update(kv_start=kv_start.int().cuda(), q=randn(rows, H, c["Dn"] + c["P"]), kv=randn(total, H, c["Dn"] + c["Dv"]),
             key=randn(total, c["P"]), out=torch.empty(rows, H, c["Dv"], dtype=dt, device="cuda"),
             spans=list(zip(start.tolist(), new.tolist(), kv_start.tolist(), lens.tolist())),
             scale=float(c["Dn"] + c["P"]) ** -0.5)
    return s


def work(case):
    c = case
    e = 4 if c["src"] == "f32" else 2
    if c["op"] == "rope":
        n = c["N"] * (c["Hq"] + c["Hkv"])
        return dict(bytes=n * c["D"] * 2 * e + c["N"] * 4, flops=n * c["rot"] * 3)
    if c["op"] == "rope_cache":
        n = c["N"] * (c["Hq"] + c["Hkv"])
        return dict(bytes=(n + c["N"] * c["Hkv"]) * c["D"] * 2 * e + c["N"] * 12, flops=n * c["rot"] * 3)
    if c["op"] == "latent_append":
        return dict(bytes=c["N"] * (c["R"] + c["P"] + c["H"] * c["P"]) * 2 * e + c["N"] * 12,
                    flops=c["N"] * (c["H"] + 1) * c["P"] * 3)
    L = (c["ctx_min"] + c["ctx_max"]) / 2.0
    n = (c["new_min"] + c["new_max"]) / 2.0
    if c["op"] == "latent_decode":
        R, P, H = c["R"], c["P"], c["H"]
        return dict(bytes=c["B"] * e * (L * (R + P) + n * H * (2 * R + P)),
                    flops=2.0 * c["B"] * H * n * max(1.0, L - n / 2) * (2 * R + P))
    d = c["Dn"] + c["P"] + c["Dv"]
    return dict(bytes=c["B"] * e * (L * (c["H"] * (c["Dn"] + c["Dv"]) + c["P"]) + n * c["H"] * d),
                flops=2.0 * c["B"] * c["H"] * n * max(1.0, L - n / 2) * d)


# ----------------------------------------------------------------- plain forms

def _frequencies(c):
    """Radians a position of each pair, in 64 bits, and the factor on the result."""
    d = c.get("rot", c.get("P"))
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    s = YARN["factor"]
    if c["scaling"] == "ntk":
        return torch.pow(BASE * s ** (d / (d - 2)), -2 * i / d), 1.0
    f = torch.pow(BASE, -2 * i / d)
    if c["scaling"] == "none":
        return f, 1.0
    if c["scaling"] == "linear":
        return f / s, 1.0

    def pair(turns):                 # the pair that makes so many turns over the original length
        return d * math.log(YARN["original"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))

    lo, hi = max(0, math.floor(pair(YARN["beta_fast"]))), min(d - 1, math.ceil(pair(YARN["beta_slow"])))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1


def _turned(x, c, pos):
    """x [N, H, D] with its first `rot` elements rotated, in 32 bits."""
    f, amp = _frequencies(c)
    angle = pos.double()[:, None] * f[None]
    co, si = (torch.cos(angle) * amp).float()[:, None], (torch.sin(angle) * amp).float()[:, None]
    n = f.numel()
    x = x.float()
    r, rest = x[..., :2 * n], x[..., 2 * n:]
    if c["layout"] == "half":
        a, b = r[..., :n], r[..., n:]
        return torch.cat([a * co - b * si, b * co + a * si, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2), rest], -1)


def _plain_turn(s):
    c = s["case"]
    s["q_out"].copy_(_turned(s["q"], c, s["pos"]))
    if c["op"] == "rope":
        s["k_out"].copy_(_turned(s["k"], c, s["pos"]))
        return s["q_out"], s["k_out"]
    if c["op"] == "rope_cache":
        for pool, x in ((s["k_cache"], _turned(s["k"], c, s["pos"])), (s["v_cache"], s["v"])):
            pool.view(-1, c["Hkv"], c["D"])[s["slots"]] = x.to(pool.dtype)
        return s["q_out"], s["k_cache"], s["v_cache"]
    key = _turned(s["key"][:, None], c, s["pos"])[:, 0].to(s["cache"].dtype)
    s["cache"].view(-1, c["R"] + c["P"])[s["slots"]] = torch.cat([s["latent"], key], -1)
    return s["q_out"], s["cache"]


def _softmax(x):
    """Over the last axis; every row here has something in it."""
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_decode(s):
    c = s["case"]
    B, H, bs, n = c["B"], c["H"], c["bs"], s["max_new"]
    cols = -(-s["max_len"] // bs)
    t = torch.arange(cols * bs, device="cuda")
    lens, start = s["lens"].long(), s["start"].long()
    new = start[1:] - start[:-1]
    ids = s["table"][:, :cols].long()
    ids = torch.where(t[::bs][None] < lens[:, None], ids, torch.zeros_like(ids))
    C = s["cache"][ids].float().view(B, cols * bs, -1)
    C = torch.where((t[None] < lens[:, None])[..., None], C, torch.zeros((), device="cuda"))
    i = torch.arange(n, device="cuda")
    row = (start[:-1, None] + i[None]).clamp(max=s["rows"] - 1)
    q = s["q"][row].float().view(B, n * H, -1)
    x = (torch.matmul(q, C.transpose(1, 2)) * s["scale"]).view(B, n, H, -1)
    # a row past the sequence's own sees its whole context and is dropped below
    at = torch.minimum((lens - new)[:, None] + i[None], lens[:, None] - 1)
    x = torch.where(t[None, None] <= at[..., None], x.transpose(1, 2).transpose(0, 1),
                    torch.full((), -math.inf, device="cuda")).permute(1, 2, 0, 3)
    o = torch.matmul(_softmax(x).reshape(B, n * H, -1), C[..., :c["R"]]).view(B, n, H, -1)
    return o[i[None] < new[:, None]].to(s["q"].dtype)


def _plain_prefill(s):
    c = s["case"]
    H, Dn = c["H"], c["Dn"]
    for q0, n, k0, L in s["spans"]:
        q, kv = s["q"][q0:q0 + n].float().transpose(0, 1), s["kv"][k0:k0 + L].float().transpose(0, 1)
        key = torch.cat([kv[..., :Dn], s["key"][k0:k0 + L].float()[None].expand(H, L, -1)], -1)
        see = torch.arange(L, device="cuda")[None] <= torch.arange(L - n, L, device="cuda")[:, None]
        x = torch.matmul(q, key.transpose(1, 2)) * s["scale"]
        x = torch.where(see[None], x, torch.full((), -math.inf, device="cuda"))
        s["out"][q0:q0 + n] = torch.matmul(_softmax(x), kv[..., Dn:]).transpose(0, 1).to(s["out"].dtype)
    return s["out"]


# -------------------------------------------------------------------------- run

def run(state):
    s = state
    if own:
        return _own(s)
    if s["case"]["op"] == "latent_decode":
        return _plain_decode(s)
    if s["case"]["op"] == "latent_prefill":
        return _plain_prefill(s)
    return _plain_turn(s)


def _own(s):
    from paged_kv_cache_307_gb300 import _lib as pa
    c = s["case"]
    op = c["op"]
    if op == "latent_prefill":
        return pa.latent_prefill(s["out"], s["q"], s["start"], s["kv"], s["key"], s["kv_start"], s["scale"])
    if op == "latent_decode":
        start = s["start"] if c["new_max"] > 1 else None
        if "workspace" not in s:         # a serving program keeps it from step to step
            s["workspace"] = pa.alloc_latent_workspace(s["q"], s["cache"], s["table"])
        return pa.latent_decode(s["out"], s["q"], s["cache"], s["table"], s["lens"], s["scale"], query_start=start,
                                workspace=s["workspace"])
    if "steps" not in s:                 # a model's constant
        kw = {} if c["scaling"] == "none" else dict(factor=YARN["factor"])
        if c["scaling"] == "yarn":
            kw.update(original_len=YARN["original"], beta_fast=YARN["beta_fast"], beta_slow=YARN["beta_slow"])
        s["steps"] = pa.rope_steps(c.get("rot", c.get("P")), BASE, scaling=c["scaling"], device="cuda", **kw)
    turn = dict(layout=c["layout"], amplitude=s["steps"][1])
    if op == "rope":
        return pa.rope(s["q"], s["k"], s["pos"], s["steps"][0], q_out=s["q_out"], k_out=s["k_out"], **turn)
    if op == "rope_cache":
        pa.rope_and_cache(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_cache"], s["v_cache"], s["steps"][0],
                          q_out=s["q_out"], **turn)
        return s["q_out"], s["k_cache"], s["v_cache"]
    pa.latent_append(s["latent"], s["key"], s["pos"], s["slots"], s["cache"], s["steps"][0], query=s["q"],
                     query_out=s["q_out"], **turn)
    return s["q_out"], s["cache"]


# ------------------------------------------------- the definitions, in 64 bits

def _f64_frequency(c, i):
    d = c.get("rot", c.get("P"))
    f = BASE ** (-2.0 * i / d)
    s = YARN["factor"]
    if c["scaling"] == "linear":
        return f / s
    if c["scaling"] == "ntk":
        return (BASE * s ** (d / (d - 2.0))) ** (-2.0 * i / d)
    if c["scaling"] == "yarn":
        edge = [d * math.log(YARN["original"] / (2 * math.pi * YARN[b])) / (2 * math.log(BASE))
                for b in ("beta_fast", "beta_slow")]
        lo, hi = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
        part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
        return f * (part / s + 1 - part)
    return f


def _f64_turned(x, c, pos):
    """Each pair as a complex number, times amplitude e^(i position frequency)."""
    d = c.get("rot", c.get("P"))
    f = torch.tensor([_f64_frequency(c, i) for i in range(d // 2)], dtype=torch.float64, device="cuda")
    amp = 0.1 * math.log(YARN["factor"]) + 1 if c["scaling"] == "yarn" else 1.0
    turn = torch.polar(torch.full((), amp, dtype=torch.float64, device="cuda").expand(len(pos), d // 2).contiguous(),
                       pos.double()[:, None] * f)[:, None]
    y = x.double().clone()
    first, second = ((slice(0, d // 2), slice(d // 2, d)) if c["layout"] == "half" else
                     (slice(0, d, 2), slice(1, d, 2)))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("rope", "rope_cache", "latent_append"):
        q = _f64_turned(s["q"], c, s["pos"])
        if c["op"] == "rope":
            return q, _f64_turned(s["k"], c, s["pos"])
        bs = c["bs"]
        block, slot = s["slots"] // bs, s["slots"] % bs
        if c["op"] == "rope_cache":
            k, v = s["k_cache"].double(), s["v_cache"].double()
            k[block, slot], v[block, slot] = _f64_turned(s["k"], c, s["pos"]), s["v"].double()
            return q, k, v
        cache = s["cache"].double()
        cache[block, slot, :c["R"]] = s["latent"].double()
        cache[block, slot, c["R"]:] = _f64_turned(s["key"][:, None], c, s["pos"])[:, 0]
        return q, cache
    if work(c)["flops"] > 4e12:
        return None                      # over 20 seconds in 64 bits
    lens, start = s["lens"].tolist(), s["start"].tolist()
    outs = []
    for b, L in enumerate(lens):
        n = start[b + 1] - start[b]
        q = s["q"][start[b]:start[b + 1]].double()
        late = torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None]
        if c["op"] == "latent_decode":
            ids = s["table"][b, :-(-L // c["bs"])].long()
            C = s["cache"][ids].double().reshape(-1, c["R"] + c["P"])[:L]
            x = torch.einsum("nhd,td->hnt", q, C) * s["scale"]
            outs.append(torch.einsum("hnt,td->nhd", torch.softmax(x.masked_fill(late, -math.inf), -1), C[:, :c["R"]]))
            continue
        k0 = int(s["kv_start"][b])
        kv, key = s["kv"][k0:k0 + L].double(), s["key"][k0:k0 + L].double()
        o = torch.empty(n, c["H"], c["Dv"], dtype=torch.float64, device="cuda")
        for h in range(c["H"]):
            x = (q[:, h, :c["Dn"]] @ kv[:, h, :c["Dn"]].T + q[:, h, c["Dn"]:] @ key.T) * s["scale"]
            o[:, h] = torch.softmax(x.masked_fill(late, -math.inf), -1) @ kv[:, h, c["Dn"]:]
        outs.append(o)
    return torch.cat(outs)
