"""What the rotary calls and the calls of the latent cache refuse, on the host (CPU only: nothing below reaches a
launch)."""

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


def _steps(pa, out=True, d=64, base=1e4, kind=0, factor=2.0, length=4096.0, fast=32.0, slow=1.0):
    t, a = (ctypes.c_uint64 * 256)(), ctypes.c_float()
    return pa.lib.pa_rope_steps(t if out else None, ctypes.byref(a), d, base, kind, factor, length, fast, slow)


def _rope(pa, qo=FAKE, q=FAKE, qs=4096, qh=128, Hq=4, ko=FAKE, k=FAKE, ks=1024, Hk=2, pos=FAKE, n=3, D=128, rot=128, lay=0,
          steps=FAKE, dt=1):
    return pa.lib.pa_rope(qo, 512, 128, q, qs, qh, Hq, ko, 256, 128, k, ks, 128, Hk, pos, n, D, rot, lay, steps, 1.0, dt,
                          NULL)


def _cache(pa, q=FAKE, Hq=4, key=FAKE, ks=256, value=FAKE, H=2, slots=FAKE, n=3, kc=FAKE, NB=4, bs=16, D=128, rot=64,
           lay=1, steps=FAKE, dt=1):
    return pa.lib.pa_rope_and_cache(FAKE, 512, 128, q, 512, 128, Hq, key, ks, 128, value, 256, 128, H, FAKE, slots, n, kc,
                                    FAKE, NB, bs, D, rot, lay, steps, 1.0, dt, NULL)


def _append(pa, lat=FAKE, ls=512, key=FAKE, ks=64, q=FAKE, qh=64, H=4, slots=FAKE, n=3, cache=FAKE, NB=4, bs=16, R=512,
            P=64, lay=0, dt=1):
    return pa.lib.pa_latent_append(lat, ls, key, ks, FAKE, 256, 64, q, 256, qh, H, FAKE, slots, n, cache, NB, bs, R, P, lay,
                                   FAKE, 1.0, dt, NULL)


def _decode(pa, q=FAKE, start=NULL, rows=2, cache=FAKE, mb=4, B=2, H=16, R=512, P=64, bs=16, NB=10, scale=1.0,
            ws=FAKE, n=1 << 40, dt=1):
    return pa.lib.pa_latent_decode(FAKE, q, start, rows, cache, FAKE, mb, FAKE, B, H, R, P, bs, NB, scale, ws, n, dt,
                                   NULL)


def _prefill(pa, q=FAKE, start=FAKE, rows=4, kv=FAKE, key=FAKE, ks=64, T=8, B=2, H=4, Dk=128, P=64, Dv=128, scale=1.0,
             dt=1):
    return pa.lib.pa_latent_prefill(FAKE, q, start, rows, kv, key, ks, FAKE, T, B, H, Dk, P, Dv, scale, dt, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(kind=3), 0), (dict(d=0), -2), (dict(d=24), -2), (dict(d=528), -2), (dict(base=1.0), -2),
    (dict(base=float("nan")), -2), (dict(kind=4), -2), (dict(kind=-1), -2), (dict(kind=1, factor=0.5), -2), (dict(kind=0, factor=0.5), 0),
    (dict(kind=2, factor=float("inf")), -2), (dict(kind=3, length=0.0), -2), (dict(kind=3, slow=0.0), -2),
    (dict(kind=3, fast=0.5), -2), (dict(out=False), -1)])
def test_steps(pa, kw, code):
    assert _steps(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), -3), (dict(dt=9), -3), (dict(n=-1), -2), (dict(Hq=-1), -2), (dict(Hk=(1 << 20) + 1), -2), (dict(D=72), -2), (dict(D=528, rot=64), -2),
    (dict(rot=0), -2), (dict(rot=40), -2), (dict(rot=144), -2), (dict(lay=2), -2), (dict(q=NULL), -1),
    (dict(ko=NULL), -1), (dict(pos=NULL), -1), (dict(steps=NULL), -1), (dict(qo=ODD), -4), (dict(k=ODD), -4),
    (dict(qs=4100), -4), (dict(qh=132), -4), (dict(ks=1026, dt=0), -4), (dict(n=0, q=NULL), 0), (dict(Hq=0, Hk=0, q=NULL), 0)])
def test_rope(pa, kw, code):
    assert _rope(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), -3), (dict(D=48, rot=48), -2), (dict(D=256), -2), (dict(bs=12), -2), (dict(NB=0), -2), (dict(H=0), -2),
    (dict(rot=24), -2), (dict(lay=-1), -2), (dict(n=-1), -2), (dict(key=NULL), -1), (dict(value=NULL), -1),
    (dict(slots=NULL), -1), (dict(kc=NULL), -1), (dict(steps=NULL), -1), (dict(q=NULL), -1), (dict(q=ODD), -4), (dict(key=ODD), -4),
    (dict(ks=260), -4), (dict(kc=ODD), -4), (dict(n=0, key=NULL), 0)])
def test_rope_and_cache(pa, kw, code):
    assert _cache(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), -3), (dict(R=500), -2), (dict(R=640), -2), (dict(R=0), -2), (dict(P=80), -2), (dict(P=24), -2), (dict(P=0), -2), (dict(bs=4), -2),
    (dict(bs=64), -2), (dict(NB=0), -2), (dict(lay=3), -2), (dict(n=-1), -2), (dict(H=-1), -2), (dict(lat=NULL), -1), (dict(key=NULL), -1),
    (dict(q=NULL), -1), (dict(slots=NULL), -1), (dict(cache=NULL), -1), (dict(lat=ODD), -4), (dict(ls=514), -4), (dict(ks=68), -4),
    (dict(qh=68), -4), (dict(cache=ODD), -4), (dict(n=0, lat=NULL), 0)])
def test_latent_append(pa, kw, code):
    assert _append(pa, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), -3), (dict(dt=2), -3), (dict(R=192), -2), (dict(R=640), -2), (dict(P=72), -2), (dict(P=0), -2), (dict(bs=4), -2), (dict(bs=64), -2),
    (dict(H=0), -2), (dict(rows=3), -2), (dict(rows=-1, start=FAKE), -2), (dict(NB=0), -2), (dict(mb=0), -2), (dict(mb=(1 << 25) + 1, bs=32), -2),
    (dict(scale=0.0), -2), (dict(scale=float("nan")), -2), (dict(rows=1 << 28, B=1 << 28, H=16), -2),
    (dict(q=NULL), -1), (dict(cache=NULL), -1), (dict(q=ODD), -4), (dict(cache=ODD), -4), (dict(ws=ODD), -4), (dict(ws=NULL), -5),
    (dict(n=100), -5), (dict(B=0, rows=0), 0),
    (dict(rows=0, start=FAKE, q=NULL), 0)])
def test_latent_decode(pa, kw, code):
    assert _decode(pa, **kw) == code


def test_latent_decode_of_too_many_tiles(pa):
    """Row groups and tiles are counted in 31 bits: (rows / 16 + sequences) x tiles of a table row."""
    assert _decode(pa, mb=1 << 26, bs=16, rows=128, B=128) == -2
    assert _decode(pa, mb=1 << 26, bs=16, rows=127, B=127, n=0) == -5      # (in range: the workspace is looked at next)
    assert _decode(pa, mb=1 << 20, bs=16, rows=1 << 14, B=1 << 14) == -2


def test_latent_decode_of_too_many_tiles_for_wider_groups(pa):
    """The same by groups of 32 and 64 rows: 2^14 and 2^15 tiles a table row, on each side of the limit (the
    workspace is looked at next)."""
    assert _decode(pa, mb=1 << 17, H=32, rows=1 << 16, B=1 << 16, n=0) == -2              # (2^16 + 2^16) x 2^14
    assert _decode(pa, mb=1 << 17, H=32, rows=(1 << 16) - 1, B=(1 << 16) - 1, n=0) == -5
    # 64 rows a sequence or more: rows x 128 heads / 64 and the sequences
    assert _decode(pa, mb=1 << 18, H=128, rows=3 * 21846, start=FAKE, B=3, n=0) == -2     # 131079 groups
    assert _decode(pa, mb=1 << 17, H=128, rows=65534, start=FAKE, B=3, n=0) == -5         # 131071 x 2^14
    assert _decode(pa, mb=1 << 17, H=64, rows=65536, start=FAKE, B=65536, n=0) == -2      # 131072 x 2^14
    assert _decode(pa, mb=1 << 17, H=64, rows=65535, start=FAKE, B=65535, n=0) == -5


def test_workspace_arithmetic(pa):
    need = pa.lib.pa_latent_decode_workspace_bytes
    # two slots a CTA of 152: 16 or 64 rows of 512 sums, their maxima and sums, 16 bytes a slot
    assert need(4, 4, 16, 512) == 2 * 152 * (16 * (512 * 4 + 8) + 16)
    assert need(4, 4, 128, 512) == 2 * 152 * (64 * (512 * 4 + 8) + 16)
    assert need(0, 4, 16, 512) == need(4, 0, 16, 512) == need(4, 4, 16, 500) == need(-1, 4, 16, 512) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), -3), (dict(dt=2), -3), (dict(Dk=96), -2), (dict(Dk=256), -2), (dict(Dv=16), -2), (dict(P=0), -2), (dict(P=72), -2),
    (dict(H=0), -2), (dict(rows=-1), -2), (dict(T=-1), -2), (dict(B=-1), -2), (dict(B=2049), -2), (dict(ks=56), -2), (dict(scale=-1.0), -2),
    (dict(scale=float("nan")), -2), (dict(rows=1 << 30), -2), (dict(q=NULL), -1), (dict(start=NULL), -1), (dict(kv=NULL), -1), (dict(key=NULL), -1),
    (dict(q=ODD), -4), (dict(kv=ODD), -4), (dict(key=ODD), -4), (dict(ks=68), -4), (dict(B=0), 0), (dict(rows=0, q=NULL), 0)])
def test_latent_prefill(pa, kw, code):
    assert _prefill(pa, **kw) == code


# ---------------------------------------------------------------- the binding's own checks

def _refuses(f, ok, *changes):
    for change in changes + ({},):                               # (the last all in order, but on the CPU)
        with pytest.raises((ValueError, TypeError)):
            f(**dict(ok, **change))


def test_binding_refuses_wrong_tensors(pa):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)         # noqa: E731
    pos, slots, steps = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(16, dtype=torch.int64)
    q, k = bf(3, 4, 64), bf(3, 2, 64)
    _refuses(pa.rope, dict(q=q, k=k, positions=pos, steps=steps),
             dict(q=None, k=None), dict(q=q.half(), k=None), dict(k=k.float()), dict(k=bf(3, 2, 32)), dict(k=k[:2]),
             dict(q=q.transpose(1, 2)), dict(positions=pos.long()), dict(positions=pos[:2]), dict(steps=steps.int()),
             dict(layout="quarter"), dict(q_out=bf(3, 4, 32)), dict(q_out=bf(1, 4, 64).expand(3, 4, 64)),
             dict(q=bf(3, 1, 64).expand(3, 4, 64)), dict(k=None, k_out=k))
    pool = bf(4, 16, 2, 64)
    _refuses(pa.rope_and_cache, dict(q=q, key=k, value=k, positions=pos, slot_mapping=slots, k_cache=pool, v_cache=pool.clone(),
                                     steps=steps),
             dict(key=k.float()), dict(value=bf(3, 3, 64)), dict(q=bf(3, 4, 32)), dict(slot_mapping=pos), dict(q=q[:2]),
             dict(v_cache=bf(4, 16, 2, 32)), dict(k_cache=pool.byte(), v_cache=pool.byte()), dict(slot_mapping=slots[:2]))
    cache, steps = bf(4, 16, 576), torch.zeros(32, dtype=torch.int64)
    _refuses(pa.latent_append, dict(latent=bf(3, 512), key_rope=bf(3, 64), positions=pos, slot_mapping=slots, cache=cache, steps=steps,
                                    query=q),
             dict(latent=bf(3, 256)), dict(latent=torch.zeros(3, 512)), dict(key_rope=bf(64, 3).T), dict(steps=steps[:16]), dict(query=bf(3, 4, 32)),
             dict(cache=bf(4, 16, 2, 288)), dict(query=bf(2, 4, 64)), dict(key_rope=bf(2, 64)))
    tab, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    _refuses(pa.latent_decode, dict(out=bf(2, 4, 512), q=bf(2, 4, 576), cache=cache, block_tables=tab, context_lens=lens, scale=1.0),
             dict(q=bf(2, 4, 512)), dict(q=bf(3, 4, 576), out=bf(3, 4, 512)), dict(out=bf(2, 3, 512)), dict(out=torch.zeros(2, 4, 512)),
             dict(query_start=torch.zeros(2, dtype=torch.int32)), dict(context_lens=lens[:1]), dict(block_tables=tab.long()))
    st = torch.tensor([0, 1, 3], dtype=torch.int32)
    _refuses(pa.latent_prefill, dict(out=bf(3, 4, 128), q=bf(3, 4, 192), query_start=st, kv=bf(5, 4, 256), key_rope=bf(5, 64), kv_start=st,
                                     scale=1.0),
             dict(kv=bf(5, 4, 192)), dict(kv=bf(4, 4, 256)), dict(q=bf(3, 3, 192)), dict(out=torch.zeros(3, 4, 128)), dict(kv_start=st[:2]),
             dict(query_start=st.long()), dict(key_rope=bf(64, 5).T))
    with pytest.raises(ValueError):
        pa.rope_steps(64, scaling="other")
    with pytest.raises(pa.PAError):
        pa.rope_steps(60)
    with pytest.raises(pa.PAError):
        pa.rope_steps(-16)
