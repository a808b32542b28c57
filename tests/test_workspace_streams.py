"""The workspace that a call makes for itself belongs to the stream that the call runs on: memory that the current
stream has freed, but may still be writing, is not handed to it."""

import contextlib

import pytest
import torch

from paged_kv_cache_307_gb300 import build as B


@pytest.fixture(scope="module")
def pa():
    B.build()
    from paged_kv_cache_307_gb300 import _lib
    return _lib


class _Lib:
    """Workspaces of 4096 bytes, and calls that do nothing."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_bytes") else 0


class _Stream:
    cuda_stream = 0x1234


def _calls(pa, stream):
    """Every call that makes a workspace, as (name, function), over small host tensors."""
    B_, Hq, Hkv, D, bs, cols, NB = 2, 4, 2, 64, 16, 3, 8
    i32 = dict(dtype=torch.int32)
    q, out = torch.zeros(B_, Hq, D, dtype=torch.bfloat16), torch.zeros(B_, Hq, D, dtype=torch.bfloat16)
    k, v = (torch.zeros(NB, bs, Hkv, D, dtype=torch.bfloat16) for _ in range(2))
    k8, v8 = (torch.zeros(NB, bs, Hkv, D, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.ones(NB, 4) for _ in range(2))
    ts = torch.ones(NB, bs)
    tab, lens = torch.zeros(B_, cols, **i32), torch.ones(B_, **i32)
    w, pos = torch.zeros(B_, Hkv, cols * bs), torch.zeros(B_, Hkv, cols * bs, **i32)
    at = dict(stream=stream)
    return [
        ("decode", lambda: pa.decode(out, q, k, v, tab, lens, 1.0, **at)),
        ("decode_shared", lambda: pa.decode_shared(out, q, k, v, tab, lens, torch.tensor([0, 2], **i32),
                                                   torch.tensor([1], **i32), 1.0, **at)),
        ("decode_fp8", lambda: pa.decode_fp8(out, q, k8, v8, ts, ts, tab, lens, 1.0, **at)),
        ("decode_fp8_blocks", lambda: pa.decode_fp8_blocks(out, q, k8, v8, ks, vs, tab, lens, 1.0, **at)),
        ("decode_weights", lambda: pa.decode_weights(out, w, q, k, v, tab, lens, 1.0, **at)),
        ("evict", lambda: pa.evict(k, v, tab, lens, lens, lens, w, pos, 8, lens, w, pos, **at)),
    ]


NAMES = ["decode", "decode_shared", "decode_fp8", "decode_fp8_blocks", "decode_weights", "evict"]


@pytest.mark.parametrize("name", NAMES)
def test_workspace_is_allocated_on_the_calls_stream(pa, name, monkeypatch):
    current, made = [None], []
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def record(*a, **kw):
        made.append(current[-1])
        return empty(*a, **kw)

    mine = _Stream()
    run = dict(_calls(pa, mine))[name]
    monkeypatch.setattr(pa, "lib", _Lib())
    monkeypatch.setattr(pa, "_ready", lambda *ts: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", record)
    run()
    assert made == [mine]


@pytest.mark.gpu
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_decode_beside_writes_to_memory_the_current_stream_freed(pa, pool):
    """The current stream still writes a tensor of the workspace's size, freed on the host, while the call runs
    on another stream."""
    from _bounded import Case, check, reference
    c = Case(pool, [3000] * 8, 8, 2, 128, 16, seed=2)
    ref, tol = reference(c)
    c.cuda()
    out = torch.empty_like(c.q)
    side = torch.cuda.Stream()
    if pool == "bf16":
        n = pa.alloc_workspace(c.q, c.k, c.tab).numel()
        run = lambda: pa.decode(out, c.q, c.k, c.v, c.tab, c.lens, c.scale, stream=side)      # noqa: E731
    else:
        n = pa.alloc_fp8_blocks_workspace(c.q, c.k, c.tab).numel()
        run = lambda: pa.decode_fp8_blocks(out, c.q, c.k, c.v, c.ks, c.vs, c.tab, c.lens, c.scale,   # noqa: E731
                                           stream=side)
    assert n > 16
    torch.cuda.synchronize()
    assert pa.last_error() == 0
    for _ in range(5):
        freed = torch.empty(n, dtype=torch.uint8, device="cuda")
        for _ in range(300):
            freed.fill_(0x7F)
        del freed
        for _ in range(20):
            run()
    torch.cuda.synchronize()
    assert pa.last_error() == 0
    check(out, ref, tol)
