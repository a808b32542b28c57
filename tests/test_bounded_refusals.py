"""What the calls of the block-scaled cache, the weight-keeping decode and the eviction refuse, on the host
(CPU only: nothing below reaches a launch)."""

import ctypes

import pytest
import torch

from paged_kv_cache_307_gb300 import build as B

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)        # never dereferenced: every call is rejected first
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def pa():
    B.build()
    from paged_kv_cache_307_gb300 import _lib
    return _lib


def _append(pa, key=FAKE, T=4, mb=8, B=2, k_scale=FAKE, NB=10, bs=16, H=2, D=64, dt=1):
    return pa.lib.pa_append_fp8_blocks(key, FAKE, FAKE, T, FAKE, mb, FAKE, B, FAKE, FAKE, k_scale, FAKE, NB, bs, H, D,
                                       dt, NULL)


def _decode(pa, q=FAKE, ks=FAKE, mb=4, B=2, Hq=8, H=2, D=128, bs=16, ps=0, ws=NULL, n=0, dt=1):
    return pa.lib.pa_decode_fp8_blocks(FAKE, q, FAKE, FAKE, ks, FAKE, FAKE, mb, FAKE, B, Hq, H, D, bs, 10, 1.0, ps, ws,
                                       n, dt, NULL)


def _prefill(pa, q=FAKE, start=FAKE, T=4, ks=FAKE, mb=4, B=2, Hq=8, H=2, D=128, bs=16, scale=1.0, dt=1):
    return pa.lib.pa_prefill_fp8_blocks(FAKE, q, start, T, FAKE, FAKE, ks, FAKE, FAKE, mb, FAKE, B, Hq, H, D, bs, 10,
                                        scale, dt, NULL)


def _weights(pa, w=FAKE, stride=64, ks=FAKE, B=2, Hq=8, H=2, D=128, bs=16, mb=4, ws=FAKE, n=1 << 40, dt=1, kv=1):
    return pa.lib.pa_decode_weights(FAKE, w, stride, FAKE, FAKE, FAKE, ks, FAKE, FAKE, mb, FAKE, B, Hq, H, D, bs, 10,
                                    1.0, 0, ws, n, dt, kv, NULL)


def _evict(pa, k=FAKE, ks=FAKE, mb=4, B=2, budget=32, recent=8, sinks=2, stride=64, bs=16, H=2, D=64, ws=FAKE,
           n=1 << 40, kv=1, new=FAKE):
    return pa.lib.pa_evict(k, FAKE, ks, FAKE, FAKE, mb, FAKE, FAKE, FAKE, B, FAKE, FAKE, budget, recent, sinks, new,
                           FAKE, FAKE, stride, 10, bs, H, D, ws, n, kv, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(D=48), -2), (dict(bs=12), -2), (dict(H=0), -2), (dict(T=-1), -2), (dict(B=-1), -2), (dict(NB=0), -2),
    (dict(mb=0), -2), (dict(mb=1 << 28, bs=32), -2), (dict(mb=(1 << 25) + 1, bs=32), -2), (dict(H=1 << 20), -2), (dict(dt=2), -3), (dict(dt=9), -3),
    (dict(k_scale=NULL), -1), (dict(key=NULL), -1), (dict(key=ODD), -4), (dict(k_scale=ODD), -4),
    (dict(T=0, key=NULL), 0), (dict(B=0), 0)])
def test_append(pa, kw, code):
    assert _append(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), -3), (dict(dt=2), -3), (dict(D=96), -2), (dict(Hq=7), -2), (dict(bs=64), -2), (dict(ps=24), -2), (dict(mb=(1 << 25) + 1, bs=32), -2),
    (dict(ks=NULL), -1), (dict(q=NULL), -1), (dict(ks=ODD), -4), (dict(q=ODD), -4),
    (dict(mb=64, ps=512), -5), (dict(mb=64, ps=512, ws=FAKE, n=16), -5), (dict(mb=64, ps=512, ws=ODD, n=1 << 30), -4),
    (dict(B=0), 0)])
def test_decode(pa, kw, code):
    assert _decode(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), -3), (dict(D=96), -2), (dict(Hq=7), -2), (dict(bs=2), -2), (dict(scale=0.0), -2), (dict(mb=(1 << 25) + 1, bs=32), -2),
    (dict(scale=float("nan")), -2), (dict(T=-1), -2), (dict(start=NULL), -1), (dict(ks=NULL), -1), (dict(q=ODD), -4),
    (dict(T=0, q=NULL), 0), (dict(B=0), 0)])
def test_prefill(pa, kw, code):
    assert _prefill(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(stride=63), -2), (dict(mb=(1 << 25) + 1, bs=32, stride=1 << 40), -2), (dict(Hq=2050), -2), (dict(D=40), -2), (dict(dt=0, kv=1), -3), (dict(dt=0, kv=2), -3),
    (dict(kv=5), -3), (dict(w=NULL), -1), (dict(kv=2, ks=NULL), -1), (dict(kv=2, ks=ODD), -4), (dict(ws=ODD), -4), (dict(ws=NULL), -5),
    (dict(n=100), -5), (dict(B=0), 0)])
def test_weights(pa, kw, code):
    assert _weights(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(budget=0), -2), (dict(recent=-1), -2), (dict(sinks=-1), -2), (dict(recent=20, sinks=13), -2),
    (dict(stride=63), -2), (dict(mb=393217, stride=1 << 40), -2), (dict(bs=5), -2), (dict(D=16), -2), (dict(kv=3), -3), (dict(k=NULL), -1),
    (dict(new=NULL), -1), (dict(kv=2, ks=NULL), -1), (dict(k=ODD), -4), (dict(ws=ODD), -4), (dict(ws=NULL), -5),
    (dict(n=8), -5), (dict(B=0), 0)])
def test_evict(pa, kw, code):
    assert _evict(pa, **kw) == code


def test_workspace_arithmetic(pa):
    L = pa.lib
    # 2 seqs x 8 heads, 64 slots: one partition of (m, l), the counter, a score per slot
    assert L.pa_decode_weights_workspace_bytes(2, 8, 2, 128, 4, 16, 0, 1) == 256 + 256 + 2 * 8 * 64 * 4
    # two partitions of 32 tokens: partial outputs too
    assert L.pa_decode_weights_workspace_bytes(2, 8, 2, 128, 4, 16, 32, 1) == 256 + 32 * 128 * 4 + 256 + 2 * 8 * 64 * 4
    assert L.pa_decode_weights_workspace_bytes(0, 8, 2, 128, 4, 16, 0, 1) == 0
    part, ws = L.pa_decode_fp8_blocks_partition_size, L.pa_decode_fp8_blocks_workspace_bytes
    assert part(64, 32, 8, 128, 1024, 16, 0) == 2048              # 512 CTAs x 8 partitions at capacity
    assert part(1, 32, 8, 128, 2048, 16, 0) == 512                # 8 x 64 >= 2 x 152 > 8 x 32
    assert part(1, 8, 8, 128, 8, 16, 0) == 128                    # never longer than the table
    assert part(1, 32, 8, 64, 2048, 16, 0) == 512                 # two heads a row of codes
    assert part(1, 20, 5, 64, 2048, 16, 0) == 256                 # no whole rows: CUDA cores, 5 x 128 >= 4 x 152
    assert part(1, 32, 8, 128, 2048, 16, 24) == -2 and part(1, 32, 8, 128, 2048, 16, -1) == 32768
    assert ws(1, 32, 8, 128, 2048, 16, 512) == 32 * 64 * 8 + 32 * 64 * 512 + 256
    assert ws(1, 32, 8, 128, 2048, 16, -1) == 0
    assert L.pa_evict_workspace_bytes(0, 2, 4, 16, 32) == 0
    assert L.pa_evict_workspace_bytes(2, 2, 4, 16, 0) == 0
    assert L.pa_evict_workspace_bytes(2, 2, 4, 16, 32) > 4 * 32 * 4
    # a budget that no context exceeds moves nothing
    assert L.pa_evict_workspace_bytes(2, 2, 4, 16, 64) < L.pa_evict_workspace_bytes(2, 2, 4, 16, 32)


# ---------------------------------------------------------------- the binding's own checks

def _cache(D=64, H=2, bs=16, NB=4):
    k = torch.zeros(NB, bs, H, D, dtype=torch.uint8)
    s = torch.zeros(NB, 4)
    return k, k.clone(), s, s.clone()


def _where(B=2):
    return torch.zeros(B, 3, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)


def test_binding_refuses_wrong_tensors(pa):
    k, v, ks, vs = _cache()
    tab, lens = _where()
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    start = torch.arange(3, dtype=torch.int32)
    ok = dict(key=x, value=x, query_start=start, block_tables=tab, context_lens=lens, k_cache=k, v_cache=v,
              k_scale=ks, v_scale=vs)
    for change, err in [(dict(key=x.transpose(0, 1)), ValueError), (dict(key=x.float()), ValueError),
                        (dict(k_cache=k.float()), ValueError), (dict(k_scale=ks.double()), TypeError),
                        (dict(k_scale=torch.zeros(4, 2)), ValueError), (dict(query_start=start.long()), TypeError),
                        (dict(query_start=start[:2]), ValueError), (dict(context_lens=lens[:1]), ValueError),
                        (dict(block_tables=tab.long()), TypeError), (dict(k_scale=None), (ValueError, AttributeError)),
                        ({}, ValueError)]:                       # (all in order, but on the CPU)
        with pytest.raises(err):
            pa.append_fp8_blocks(**dict(ok, **change))
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    for bad in (dict(q=q[:1].contiguous(), out=q[:1].contiguous()), dict(out=q.float()), dict(k_cache=x), {}):
        a = dict(dict(out=q.clone(), q=q, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_tables=tab,
                      context_lens=lens, scale=1.0), **bad)
        with pytest.raises((ValueError, TypeError)):
            pa.decode_fp8_blocks(**a)
        b = dict(a, query_start=start)
        if "q" not in bad:
            with pytest.raises((ValueError, TypeError)):
                pa.prefill_fp8_blocks(**b)
    w = torch.zeros(2, 2, 48)
    kf = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(weights=w.double()), dict(weights=w[0]), dict(k_scale=ks), dict(v_cache=kf.float()), {}):
        with pytest.raises((ValueError, TypeError)):
            pa.decode_weights(**dict(dict(out=q.clone(), weights=w, q=q, k_cache=kf, v_cache=kf, block_tables=tab,
                                          context_lens=lens, scale=1.0), **bad))
    p = torch.zeros(2, 2, 48, dtype=torch.int32)
    for bad in (dict(token_pos=p.long()), dict(weights=w.double()), dict(token_pos_out=p[:, :, :32].contiguous()),
                dict(new_lens=lens[:1]), dict(k_scale=ks), {}):
        with pytest.raises((ValueError, TypeError)):
            pa.evict(**dict(dict(k_cache=kf, v_cache=kf, block_tables=tab, context_lens=lens, kept_lens=lens,
                                 seen_lens=lens, weights=w, token_pos=p, budget=8, new_lens=lens.clone(),
                                 weights_out=w, token_pos_out=p), **bad))
    with pytest.raises((ValueError, TypeError)):
        pa.evict(k, v, tab, lens, lens, lens, w, p, 8, lens.clone(), w, p)          # e4m3 without scales
