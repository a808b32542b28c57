"""The sticky conditions: every unit's come back from one call, once, and looking costs one read of the device."""

import time

import pytest
import torch

from _bounded import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_307_gb300 import build
    build.build()
    from paged_kv_cache_307_gb300 import _lib
    assert torch.cuda.is_available()
    _lib.last_error()
    return _lib


def _conditions(pa):
    """(name, call, bit): a bad block or length, or a wait that runs out, in each unit of the library."""
    c = Case("bf16", [40, 40], 8, 2, 128, 16).cuda()
    e = Case("e4m3", [40, 40], 8, 2, 128, 16).cuda()
    bad = c.tab.clone()
    bad[1, 1] = -5
    long = torch.full_like(c.lens, 10 ** 6)
    ts = torch.ones(e.k.shape[:2], device="cuda")
    q8 = e.q.to(torch.bfloat16)
    out, o8 = torch.empty_like(c.q), torch.empty_like(q8)
    slots = torch.tensor([10 ** 7], device="cuda")
    one = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    new = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 2, c.tab.shape[1] * 16, device="cuda")
    pos, zero = torch.zeros(w.shape, dtype=torch.int32, device="cuda"), torch.zeros_like(c.lens)
    q4 = c.q.view(2, 1, 8, 128)
    B, S, L, T = pa.DEV_BAD_BLOCK, pa.DEV_BAD_SLOT, pa.DEV_BAD_LEN, pa.DEV_TIMEOUT
    return [
        ("cache", lambda: pa.reshape_and_cache(one, one, slots, c.k, c.v), S),
        ("decode", lambda: pa.decode(out, c.q, c.k, c.v, bad, c.lens, c.scale), B),
        ("decode e4m3", lambda: pa.decode_fp8(o8, q8, e.k, e.v, ts, ts, bad, e.lens, e.scale), B),
        ("shared", lambda: pa.decode_shared(out, c.q, c.k, c.v, bad, c.lens, torch.tensor([0, 2], dtype=torch.int32,
                                            device="cuda"), zero[:1], c.scale), B),
        ("prefill", lambda: pa.prefill(torch.empty_like(q4), q4, c.k, c.v, bad, c.lens, c.scale), B),
        ("wait", lambda: pa.selftest_bounded_wait(1000), T),
        ("append by blocks", lambda: pa.append_fp8_blocks(new, new, st, e.tab, long, e.k, e.v, e.ks, e.vs), L),
        ("decode by blocks", lambda: pa.decode_fp8_blocks(o8, q8, e.k, e.v, e.ks, e.vs, bad, e.lens, e.scale), B),
        ("prefill by blocks", lambda: pa.prefill_fp8_blocks(o8, q8, st, e.k, e.v, e.ks, e.vs, bad, e.lens, e.scale), B),
        ("weights", lambda: pa.decode_weights(out, w, c.q, c.k, c.v, bad, c.lens, c.scale), B),
        ("weights e4m3", lambda: pa.decode_weights(o8, w, q8, e.k, e.v, bad, e.lens, e.scale, k_scale=e.ks,
                                                   v_scale=e.vs), B),
        ("evict", lambda: pa.evict(c.k, c.v, c.tab, long, zero, long, w, pos, 16, torch.empty_like(zero), w, pos),
         L | B),              # (the clamped length takes in table entries that name no block)
    ]


def test_every_units_condition_comes_back_once(pa):
    for name, call, bit in _conditions(pa):
        call()
        assert pa.last_error() == bit, name
        assert pa.last_error() == 0, name


def test_conditions_of_several_units_come_together(pa):
    want = 0
    for _, call, bit in _conditions(pa):
        call()
        want |= bit
    assert pa.last_error() == want
    assert pa.last_error() == 0


def _median_us(call, n=300):
    ts = []
    for _ in range(n):
        t = time.perf_counter()
        call()
        ts.append(time.perf_counter() - t)
    return sorted(ts)[n // 2] * 1e6


def test_looking_costs_one_read_of_the_device(pa):
    """A call that waits for the device, launches one kernel and reads one word takes about as long as two reads
    of a number; a blocking read for each of the library's units took ten times one."""
    x = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    pa.last_error()
    assert _median_us(pa.last_error) < 5 * _median_us(x.item)


def test_two_threads_looking_at_once_lose_no_condition(pa):
    from concurrent.futures import ThreadPoolExecutor
    c = Case("bf16", [40, 40], 8, 2, 128, 16).cuda()
    bad = c.tab.clone()
    bad[1, 1] = -5
    out = torch.empty_like(c.q)
    with ThreadPoolExecutor(2) as two:
        for _ in range(300):
            pa.decode(out, c.q, c.k, c.v, bad, c.lens, c.scale)
            torch.cuda.synchronize()
            a, b = two.submit(pa.last_error), two.submit(pa.last_error)
            assert a.result() | b.result() == pa.DEV_BAD_BLOCK


def test_an_error_is_reported_once(pa):
    """A call that fails in CUDA (here: waiting for the device inside a capture, which ends the capture) leaves no
    error behind for the calls after it."""
    e = Case("e4m3", [40, 40], 8, 2, 128, 16).cuda()
    new = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with pytest.raises(Exception):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            with pytest.raises(pa.PAError):
                pa.last_error()
    pa.append_fp8_blocks(new, new, st, e.tab, e.lens, e.k, e.v, e.ks, e.vs)
    assert pa.last_error() == 0
