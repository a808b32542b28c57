"""ctypes binding to libpa.so: argument marshalling only.

Every step of the path runs in libpa's CUDA kernels; this module turns torch
tensors into raw device pointers and sizes, passes torch's current CUDA
stream, and raises on a non-zero return.  There is no fallback: if libpa.so
is missing the import of this module fails.
"""

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "pa.h")

if not os.path.exists(LIB_PATH):
    raise ImportError("libpa.so is not built (run paged_kv_cache_307_gb300.build.build()): " + LIB_PATH)

lib = ctypes.CDLL(LIB_PATH)

PA_F32, PA_BF16, PA_FP8_E4M3 = 0, 1, 2
DEV_BAD_BLOCK, DEV_BAD_SLOT, DEV_BAD_LEN, DEV_TIMEOUT, DEV_BAD_GROUP = 1, 2, 4, 8, 16

_p, _i, _f, _sz, _i64p, _i32p = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                                 ctypes.c_void_p, ctypes.c_void_p)

lib.pa_reshape_and_cache.argtypes = [_p, _p, _i64p, _i, _p, _p, _i, _i, _i, _i, _i, _p]
lib.pa_reshape_and_cache.restype = _i
lib.pa_decode.argtypes = [_p, _p, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _i, _p]
lib.pa_decode.restype = _i
lib.pa_decode_noalloc.argtypes = [_p, _p, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f, _i, _i, _p]
lib.pa_decode_noalloc.restype = _i
lib.pa_decode_shared.argtypes = [_p, _p, _p, _p, _i32p, _i, _i32p, _i, _i32p, _i32p, _i, _i, _i, _i, _i, _i, _f, _i,
                                 _p, _sz, _i, _p]
lib.pa_decode_shared.restype = _i
lib.pa_decode_shared_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_shared_workspace_bytes.restype = _sz
lib.pa_decode_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_workspace_bytes.restype = _sz
lib.pa_decode_partition_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_partition_size.restype = _i
lib.pa_decode_fp8_partition_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_fp8_partition_size.restype = _i
lib.pa_copy_blocks.argtypes = [_p, _p, _i64p, _i, _i, _i, _i, _i, _i, _p]
lib.pa_copy_blocks.restype = _i
lib.pa_prefill_paged.argtypes = [_p, _p, _i, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f, _i, _p]
lib.pa_prefill_paged.restype = _i
lib.pa_reshape_and_cache_fp8.argtypes = [_p, _p, _i64p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p]
lib.pa_reshape_and_cache_fp8.restype = _i
lib.pa_decode_fp8.argtypes = [_p, _p, _p, _p, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz,
                              _i, _p]
lib.pa_decode_fp8.restype = _i
lib.pa_prefill_varlen.argtypes = [_p, _p, _i32p, _i, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f, _i, _p]
lib.pa_prefill_varlen.restype = _i
lib.pa_swap_blocks.argtypes = [_p, _p, _i, _p, _p, _i, _i64p, _i, _i, _i, _i, _i, _p]
lib.pa_swap_blocks.restype = _i
lib.pa_append_fp8_blocks.argtypes = [_p, _p, _i32p, _i, _i32p, _i, _i32p, _i, _p, _p, _p, _p, _i, _i, _i, _i, _i, _p]
lib.pa_append_fp8_blocks.restype = _i
lib.pa_decode_fp8_blocks.argtypes = lib.pa_decode_fp8.argtypes
lib.pa_decode_fp8_blocks.restype = _i
lib.pa_decode_fp8_blocks_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_fp8_blocks_workspace_bytes.restype = _sz
lib.pa_decode_fp8_blocks_partition_size.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_fp8_blocks_partition_size.restype = _i
lib.pa_prefill_fp8_blocks.argtypes = [_p, _p, _i32p, _i, _p, _p, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f,
                                      _i, _p]
lib.pa_prefill_fp8_blocks.restype = _i
lib.pa_decode_weights.argtypes = [_p, _p, ctypes.c_longlong, _p, _p, _p, _p, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i,
                                  _i, _f, _i, _p, _sz, _i, _i, _p]
lib.pa_decode_weights.restype = _i
lib.pa_decode_weights_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i]
lib.pa_decode_weights_workspace_bytes.restype = _sz
lib.pa_evict.argtypes = [_p, _p, _p, _p, _i32p, _i, _i32p, _i32p, _i32p, _i, _p, _i32p, _i, _i, _i, _i32p, _p, _i32p,
                         ctypes.c_longlong, _i, _i, _i, _i, _p, _sz, _i, _p]
lib.pa_evict.restype = _i
lib.pa_evict_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.pa_evict_workspace_bytes.restype = _sz
lib.pa_last_error.argtypes = []
lib.pa_last_error.restype = _i
lib.pa_strerror.argtypes = [_i]
lib.pa_strerror.restype = ctypes.c_char_p
lib.pa_last_host_error.argtypes = []
lib.pa_last_host_error.restype = ctypes.c_char_p
lib.pa_version.argtypes = []
lib.pa_version.restype = _i
lib.pa_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, _p]
lib.pa_selftest_bounded_wait.restype = _i


class PAError(RuntimeError):
    def __init__(self, code, what):
        extra = lib.pa_last_host_error().decode() if code == -6 else ""
        super().__init__("%s failed: %s (%d)%s" % (what, lib.pa_strerror(code).decode(), code,
                                                   (": " + extra) if extra else ""))
        self.code = code


def declared_functions():
    """Names of the functions include/pa.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pa_\w+)\s*\(", text)))


def _dtype(t):
    if t.dtype == torch.float32:
        return PA_F32
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.uint8:
        return PA_FP8_E4M3          # e4m3 codes
    raise TypeError("unsupported dtype %s" % t.dtype)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, what):
    if code != 0:
        raise PAError(code, what)


def _own(alloc, stream, *sizes):
    """A workspace of the call's own, out of the memory of the stream that the call runs on: what the current
    stream has freed it may still be writing, and what `stream` frees it has used up in its own order."""
    if stream is None:
        return alloc(*sizes)
    with torch.cuda.stream(stream):
        return alloc(*sizes)


def _contig(*ts):
    for t in ts:
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def reshape_and_cache(key, value, slot_mapping, k_cache, v_cache, stream=None):
    """Append key/value [T, Hkv, D] into the pool slots named by slot_mapping."""
    _contig(key, value, slot_mapping, k_cache, v_cache)
    NB, bs, H, D = k_cache.shape
    assert slot_mapping.dtype == torch.int64
    _check(lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(slot_mapping), key.shape[0],
                                    _ptr(k_cache), _ptr(v_cache), NB, bs, H, D, _dtype(k_cache),
                                    _stream(stream)), "pa_reshape_and_cache")


def reshape_and_cache_fp8(key, value, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Quantise key/value [T, Hkv, D] (bf16 or fp32) per token into an e4m3
    pool (uint8 codes [NB, bs, Hkv, D]) and its scales (fp32 [NB, bs])."""
    _contig(key, value, slot_mapping, k_cache, v_cache, k_scale, v_scale)
    assert k_cache.dtype == torch.uint8 and k_scale.dtype == torch.float32
    assert slot_mapping.dtype == torch.int64
    NB, bs, H, D = k_cache.shape
    assert k_scale.shape == (NB, bs) and v_scale.shape == (NB, bs)
    _check(lib.pa_reshape_and_cache_fp8(_ptr(key), _ptr(value), _ptr(slot_mapping), key.shape[0],
                                        _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), NB, bs, H, D,
                                        _dtype(key), _stream(stream)), "pa_reshape_and_cache_fp8")


def workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, block_size, partition_size=0):
    return lib.pa_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks,
                                         block_size, partition_size)


def partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, block_size, partition_size=0,
                   fp8=False):
    f = lib.pa_decode_fp8_partition_size if fp8 else lib.pa_decode_partition_size
    return f(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, block_size, partition_size)


def alloc_workspace(q, k_cache, block_tables, partition_size=0):
    B, Hq, D = q.shape
    n = workspace_bytes(B, Hq, k_cache.shape[2], D, block_tables.shape[1], k_cache.shape[1], partition_size)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, partition_size=0,
           workspace=None, stream=None):
    """out[B,Hq,D] = paged decode attention of q[B,Hq,D] over the pool."""
    _contig(out, q, k_cache, v_cache, block_tables, context_lens)
    assert block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    if workspace is None:
        workspace = _own(alloc_workspace, stream, q, k_cache, block_tables, partition_size)
    _check(lib.pa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                         block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs, NB,
                         ctypes.c_float(scale), partition_size, _ptr(workspace), workspace.numel(),
                         _dtype(q), _stream(stream)), "pa_decode")
    return out


def shared_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, block_size,
                           partition_size=0, num_groups=1):
    return lib.pa_decode_shared_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks,
                                                block_size, partition_size, num_groups)


def alloc_shared_workspace(q, k_cache, block_tables, num_groups, partition_size=0):
    B, Hq, D = q.shape
    n = shared_workspace_bytes(B, Hq, k_cache.shape[2], D, block_tables.shape[1], k_cache.shape[1],
                               partition_size, num_groups)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def decode_shared(out, q, k_cache, v_cache, block_tables, context_lens, group_start, shared_blocks, scale,
                  partition_size=0, workspace=None, stream=None):
    """out[B,Hq,D] = paged decode attention of q over the pool, reading the
    shared prompt blocks of each group (sequences group_start[g] ..
    group_start[g+1]-1 share their first shared_blocks[g] table entries)
    once for the whole group."""
    _contig(out, q, k_cache, v_cache, block_tables, context_lens, group_start, shared_blocks)
    assert block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32
    assert group_start.dtype == torch.int32 and shared_blocks.dtype == torch.int32
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    ng = shared_blocks.shape[0]
    assert group_start.shape[0] == ng + 1
    if workspace is None:
        workspace = _own(alloc_shared_workspace, stream, q, k_cache, block_tables, ng, partition_size)
    _check(lib.pa_decode_shared(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                block_tables.shape[1], _ptr(context_lens), B, _ptr(group_start),
                                _ptr(shared_blocks), ng, Hq, Hkv, D, bs, NB, ctypes.c_float(scale), partition_size,
                                _ptr(workspace), workspace.numel(), _dtype(q), _stream(stream)), "pa_decode_shared")
    return out


def decode_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
               partition_size=0, workspace=None, stream=None):
    """out[B,Hq,D] (bf16) = paged decode attention of q over an e4m3 pool."""
    _contig(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens)
    assert block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32
    assert k_cache.dtype == torch.uint8 and k_scale.dtype == torch.float32
    B, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    if workspace is None:
        workspace = _own(alloc_workspace, stream, q, k_cache, block_tables, partition_size)
    _check(lib.pa_decode_fp8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                             _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs, NB,
                             ctypes.c_float(scale), partition_size, _ptr(workspace), workspace.numel(), _dtype(q),
                             _stream(stream)), "pa_decode_fp8")
    return out


def copy_blocks_fp8(k_cache, v_cache, k_scale, v_scale, pairs, stream=None):
    """Copy-on-write for an e4m3 pool: the codes, then the scale rows."""
    copy_blocks(k_cache, v_cache, pairs, stream)
    NB, bs = k_scale.shape
    copy_blocks(k_scale.view(NB, bs, 1, 1), v_scale.view(NB, bs, 1, 1), pairs, stream)


def copy_blocks(k_cache, v_cache, pairs, stream=None):
    """Copy-on-write: block pairs[i,1] becomes a copy of block pairs[i,0]."""
    _contig(k_cache, v_cache, pairs)
    assert pairs.dtype == torch.int64
    NB, bs, H, D = k_cache.shape
    _check(lib.pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(pairs), pairs.shape[0], NB, bs, H, D,
                              _dtype(k_cache), _stream(stream)), "pa_copy_blocks")


def prefill(out, q, k_cache, v_cache, block_tables, context_lens, scale, stream=None):
    """Causal chunked-prefill tile: q/out [B, Tq, Hq, D], the last Tq tokens
    of each context."""
    _contig(out, q, k_cache, v_cache, block_tables, context_lens)
    assert block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32
    B, Tq, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    _check(lib.pa_prefill_paged(_ptr(out), _ptr(q), Tq, _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs, NB,
                                ctypes.c_float(scale), _dtype(q), _stream(stream)), "pa_prefill_paged")
    return out


def prefill_varlen(out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale, stream=None):
    """Mixed round: q/out [rows, Hq, D], sequence b's rows are
    query_start[b]..query_start[b+1]-1, the last tokens of its context."""
    _contig(out, q, query_start, k_cache, v_cache, block_tables, context_lens)
    assert query_start.dtype == torch.int32 and block_tables.dtype == torch.int32
    rows, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    B = context_lens.shape[0]
    _check(lib.pa_prefill_varlen(_ptr(out), _ptr(q), _ptr(query_start), rows, _ptr(k_cache), _ptr(v_cache),
                                 _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs,
                                 NB, ctypes.c_float(scale), _dtype(q), _stream(stream)), "pa_prefill_varlen")
    return out


def swap_blocks(dst_k, dst_v, src_k, src_v, pairs, stream=None):
    """Block pairs[i,1] of (dst_k, dst_v) becomes a copy of block pairs[i,0]
    of (src_k, src_v).  Either pool may be pinned host memory."""
    _contig(dst_k, dst_v, src_k, src_v, pairs)
    assert pairs.dtype == torch.int64 and pairs.is_cuda
    assert dst_k.shape[1:] == src_k.shape[1:] and dst_k.dtype == src_k.dtype
    _, bs, H, D = dst_k.shape
    _check(lib.pa_swap_blocks(_ptr(dst_k), _ptr(dst_v), dst_k.shape[0], _ptr(src_k), _ptr(src_v), src_k.shape[0],
                              _ptr(pairs), pairs.shape[0], bs, H, D, _dtype(dst_k), _stream(stream)),
           "pa_swap_blocks")


def scale_row(num_kv_heads):
    """Floats in one block's row of a block-scaled e4m3 cache's scales."""
    return (num_kv_heads + 3) // 4 * 4


_I32, _F32 = torch.int32, torch.float32
_KIND = {torch.float32: PA_F32, torch.bfloat16: PA_BF16, torch.uint8: PA_FP8_E4M3}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _kind(t):
    k = _KIND.get(t.dtype)
    if k is None:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return k


def _on(stream, device):
    """The raw handle of `stream`, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _ready(*ts):
    """The current device, which every tensor has to be on (the library launches there), contiguous."""
    d = torch.cuda.current_device() if ts[0].is_cuda else -2
    for t in ts:
        if t.get_device() != d or not t.is_contiguous():
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            raise ValueError("tensors must be on the current CUDA device")
    return d


def _int32(*ts):
    for t in ts:
        if t.dtype is not _I32:
            raise TypeError("lengths, tables and starts are int32")


def _table(block_tables, context_lens):
    """(num_seqs, max_blocks)"""
    _int32(block_tables, context_lens)
    shape, lens = block_tables.shape, context_lens.shape
    if len(shape) != 2 or len(lens) != 1 or lens[0] != shape[0]:
        raise ValueError("block_tables is [num_seqs, max_blocks], context_lens [num_seqs]")
    return shape


def _pools(k_cache, v_cache, k_scale=None, v_scale=None):
    """(num_blocks, block_size, num_kv_heads, head_dim, kind); an e4m3 pool comes with its block scales."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache are [num_blocks, block_size, num_kv_heads, head_dim] of one type")
    kind = _kind(k_cache)
    if kind != PA_FP8_E4M3:
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to e4m3 pools")
    else:
        if k_scale is None or v_scale is None:
            raise ValueError("a block-scaled cache needs k_scale and v_scale")
        if k_scale.dtype is not _F32 or v_scale.dtype is not _F32:
            raise TypeError("scales are float32")
        if k_scale.shape != (shape[0], scale_row(shape[2])) or v_scale.shape != k_scale.shape:
            raise ValueError("scales are [num_blocks, num_kv_heads rounded up to a multiple of 4]")
    return *shape, kind


def _block_scaled(k_cache, v_cache, k_scale, v_scale):
    sizes = _pools(k_cache, v_cache, k_scale, v_scale)
    if sizes[4] != PA_FP8_E4M3:
        raise TypeError("a block-scaled cache holds e4m3 codes in uint8 pools")
    return sizes[:4]


def _starts(query_start, num_seqs):
    _int32(query_start)
    if query_start.dim() != 1 or query_start.size(0) != num_seqs + 1:
        raise ValueError("query_start is [num_seqs + 1]")


def _query(q, out, head_dim):
    """(rows, num_heads)"""
    shape = q.shape
    if out.shape != shape or out.dtype is not q.dtype or len(shape) != 3 or shape[2] != head_dim:
        raise ValueError("q and out are [rows, num_heads, head_dim] of one type")
    return shape[0], shape[1]


def append_fp8_blocks(key, value, query_start, block_tables, context_lens, k_cache, v_cache, k_scale, v_scale,
                      stream=None):
    """Quantise key/value [T, Hkv, D] (bf16 or fp32), the last tokens of each
    context (sequence b's rows are query_start[b]..query_start[b+1]-1), into an
    e4m3 pool with one power-of-two scale per (block, KV head)."""
    NB, bs, H, D = _block_scaled(k_cache, v_cache, k_scale, v_scale)
    B, cols = _table(block_tables, context_lens)
    _starts(query_start, B)
    shape = key.shape
    if value.shape != shape or value.dtype is not key.dtype or len(shape) != 3 or shape[1] != H or shape[2] != D:
        raise ValueError("key and value are [tokens, num_kv_heads, head_dim] of one type")
    kind = _kind(key)
    dev = _ready(key, value, query_start, block_tables, context_lens, k_cache, v_cache, k_scale, v_scale)
    _check(lib.pa_append_fp8_blocks(key.data_ptr(), value.data_ptr(), query_start.data_ptr(), shape[0],
                                    block_tables.data_ptr(), cols, context_lens.data_ptr(), B, k_cache.data_ptr(),
                                    v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), NB, bs, H, D, kind,
                                    _on(stream, dev)), "pa_append_fp8_blocks")


def copy_blocks_fp8_blocks(k_cache, v_cache, k_scale, v_scale, pairs, stream=None):
    """Copy-on-write for a block-scaled e4m3 cache: the codes, then the scale rows."""
    _block_scaled(k_cache, v_cache, k_scale, v_scale)
    _ready(k_cache, v_cache, k_scale, v_scale, pairs)
    copy_blocks(k_cache, v_cache, pairs, stream)
    NB, n = k_scale.shape
    copy_blocks(k_scale.view(NB, 4, n // 4, 1), v_scale.view(NB, 4, n // 4, 1), pairs, stream)


def alloc_fp8_blocks_workspace(q, k_cache, block_tables, partition_size=0):
    """Workspace for decode_fp8_blocks with these sizes."""
    B, Hq, D = q.shape
    n = lib.pa_decode_fp8_blocks_workspace_bytes(B, Hq, k_cache.shape[2], D, block_tables.shape[1], k_cache.shape[1],
                                                 partition_size)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def decode_fp8_blocks(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                      partition_size=0, workspace=None, stream=None):
    """out[B,Hq,D] (bf16) = paged decode attention of q over a block-scaled e4m3 cache."""
    NB, bs, Hkv, D = _block_scaled(k_cache, v_cache, k_scale, v_scale)
    B, cols = _table(block_tables, context_lens)
    rows, Hq = _query(q, out, D)
    if rows != B:
        raise ValueError("one query row per sequence")
    kind = _kind(q)
    if workspace is None:
        workspace = _own(alloc_fp8_blocks_workspace, stream, q, k_cache, block_tables, partition_size)
    dev = _ready(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, workspace)
    _check(lib.pa_decode_fp8_blocks(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                    k_scale.data_ptr(), v_scale.data_ptr(), block_tables.data_ptr(), cols,
                                    context_lens.data_ptr(), B, Hq, Hkv, D, bs, NB, scale, partition_size,
                                    workspace.data_ptr(), workspace.nbytes, kind, _on(stream, dev)),
           "pa_decode_fp8_blocks")
    return out


def prefill_fp8_blocks(out, q, query_start, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                       stream=None):
    """Mixed round over a block-scaled e4m3 cache: q/out [rows, Hq, D] (bf16), sequence b's rows are
    query_start[b]..query_start[b+1]-1, the last tokens of its context, causal."""
    NB, bs, Hkv, D = _block_scaled(k_cache, v_cache, k_scale, v_scale)
    B, cols = _table(block_tables, context_lens)
    _starts(query_start, B)
    rows, Hq = _query(q, out, D)
    kind = _kind(q)
    dev = _ready(out, q, query_start, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens)
    _check(lib.pa_prefill_fp8_blocks(out.data_ptr(), q.data_ptr(), query_start.data_ptr(), rows, k_cache.data_ptr(),
                                     v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                     block_tables.data_ptr(), cols, context_lens.data_ptr(), B, Hq, Hkv, D, bs, NB,
                                     scale, kind, _on(stream, dev)), "pa_prefill_fp8_blocks")
    return out


def alloc_weights_workspace(q, k_cache, block_tables, partition_size=0):
    """Workspace for decode_weights with these sizes."""
    B, Hq, D = q.shape
    n = lib.pa_decode_weights_workspace_bytes(B, Hq, k_cache.shape[2], D, block_tables.shape[1], k_cache.shape[1],
                                              partition_size, _kind(k_cache))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def decode_weights(out, weights, q, k_cache, v_cache, block_tables, context_lens, scale, k_scale=None, v_scale=None,
                   partition_size=0, workspace=None, stream=None):
    """out[B,Hq,D] = paged decode attention of q, and weights[b,g,t] (fp32 [B, Hkv, >= max_blocks * bs]) grows by
    the softmax weights of KV head g's query heads for token t.  The pools are q's type, or a block-scaled e4m3
    cache with its scales."""
    NB, bs, Hkv, D, kv = _pools(k_cache, v_cache, k_scale, v_scale)
    B, cols = _table(block_tables, context_lens)
    rows, Hq = _query(q, out, D)
    if rows != B:
        raise ValueError("one query row per sequence")
    kind = _kind(q)
    wshape = weights.shape
    if weights.dtype is not _F32 or len(wshape) != 3 or wshape[0] != B or wshape[1] != Hkv:
        raise ValueError("weights is float32 [num_seqs, num_kv_heads, slots]")
    if workspace is None:
        workspace = _own(alloc_weights_workspace, stream, q, k_cache, block_tables, partition_size)
    ks = vs = None
    if kv == PA_FP8_E4M3:
        _ready(k_scale, v_scale)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    dev = _ready(out, weights, q, k_cache, v_cache, block_tables, context_lens, workspace)
    _check(lib.pa_decode_weights(out.data_ptr(), weights.data_ptr(), wshape[2], q.data_ptr(), k_cache.data_ptr(),
                                 v_cache.data_ptr(), ks, vs, block_tables.data_ptr(), cols, context_lens.data_ptr(),
                                 B, Hq, Hkv, D, bs, NB, scale, partition_size, workspace.data_ptr(),
                                 workspace.nbytes, kind, kv, _on(stream, dev)), "pa_decode_weights")
    return out


def alloc_evict_workspace(k_cache, block_tables, budget):
    """Workspace for evict with these sizes."""
    n = lib.pa_evict_workspace_bytes(block_tables.shape[0], k_cache.shape[2], block_tables.shape[1],
                                     k_cache.shape[1], budget)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=k_cache.device)


def evict(k_cache, v_cache, block_tables, context_lens, kept_lens, seen_lens, weights, token_pos, budget, new_lens,
          weights_out, token_pos_out, recent=0, sinks=0, k_scale=None, v_scale=None, workspace=None, stream=None):
    """Cut every (sequence, KV head) to its `budget` tokens of largest weight (protected: the first `sinks` and the
    last `recent` positions).  weights/token_pos [B, Hkv, slots] name each slot's total and position; the outputs
    may be the inputs themselves.  new_lens[b] = min(L_b, budget)."""
    NB, bs, Hkv, D, kv = _pools(k_cache, v_cache, k_scale, v_scale)
    B, cols = _table(block_tables, context_lens)
    _int32(kept_lens, seen_lens, token_pos, new_lens, token_pos_out)
    lens = context_lens.shape
    if kept_lens.shape != lens or seen_lens.shape != lens or new_lens.shape != lens:
        raise ValueError("kept_lens, seen_lens and new_lens are [num_seqs]")
    if weights.dtype is not _F32 or weights_out.dtype is not _F32:
        raise TypeError("weights are float32")
    shape = weights.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != Hkv or not (
            token_pos.shape == shape and weights_out.shape == shape and token_pos_out.shape == shape):
        raise ValueError("weights and token_pos are [num_seqs, num_kv_heads, slots], in and out alike")
    if workspace is None:
        workspace = _own(alloc_evict_workspace, stream, k_cache, block_tables, budget)
    ks = vs = None
    if kv == PA_FP8_E4M3:
        _ready(k_scale, v_scale)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    dev = _ready(k_cache, v_cache, block_tables, context_lens, kept_lens, seen_lens, weights, token_pos, new_lens,
                 weights_out, token_pos_out, workspace)
    _check(lib.pa_evict(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, block_tables.data_ptr(), cols,
                        context_lens.data_ptr(), kept_lens.data_ptr(), seen_lens.data_ptr(), B, weights.data_ptr(),
                        token_pos.data_ptr(), budget, recent, sinks, new_lens.data_ptr(), weights_out.data_ptr(),
                        token_pos_out.data_ptr(), shape[2], NB, bs, Hkv, D, workspace.data_ptr(), workspace.nbytes,
                        kv, _on(stream, dev)), "pa_evict")
    return new_lens


def selftest_bounded_wait(limit_ns, stream=None):
    """Launch the bounded-wait health check (one warp waits on an mbarrier
    nothing arrives at, giving up after ``limit_ns``)."""
    _check(lib.pa_selftest_bounded_wait(int(limit_ns), _stream(stream)), "pa_selftest_bounded_wait")


def last_error():
    """Sticky device-detected condition bits (and clear them); synchronises."""
    code = lib.pa_last_error()
    if code < 0:
        raise PAError(code, "pa_last_error")
    return code
