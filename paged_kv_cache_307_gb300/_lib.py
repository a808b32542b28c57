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
_ll, _d = ctypes.c_longlong, ctypes.c_double
_rows3 = [_p, _ll, _ll]                                  # a strided [tokens, heads, dim] tensor
lib.pa_rope_steps.argtypes = [_p, _p, _i, _d, _i, _d, _d, _d, _d]
lib.pa_rope_steps.restype = _i
lib.pa_rope.argtypes = [*_rows3, *_rows3, _i, *_rows3, *_rows3, _i, _i32p, _i, _i, _i, _i, _p, _f, _i, _p]
lib.pa_rope.restype = _i
lib.pa_rope_and_cache.argtypes = [*_rows3, *_rows3, _i, *_rows3, *_rows3, _i, _i32p, _i64p, _i, _p, _p, _i, _i, _i, _i,
                                  _i, _p, _f, _i, _p]
lib.pa_rope_and_cache.restype = _i
lib.pa_latent_append.argtypes = [_p, _ll, _p, _ll, *_rows3, *_rows3, _i, _i32p, _i64p, _i, _p, _i, _i, _i, _i, _i, _p,
                                 _f, _i, _p]
lib.pa_latent_append.restype = _i
lib.pa_latent_decode.argtypes = [_p, _p, _i32p, _i, _p, _i32p, _i, _i32p, _i, _i, _i, _i, _i, _i, _f, _p, _sz, _i, _p]
lib.pa_latent_decode.restype = _i
lib.pa_latent_decode_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.pa_latent_decode_workspace_bytes.restype = _sz
lib.pa_latent_prefill.argtypes = [_p, _p, _i32p, _i, _p, _p, _ll, _i32p, _i, _i, _i, _i, _i, _i, _f, _i, _p]
lib.pa_latent_prefill.restype = _i
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


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_steps(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=4096.0, beta_fast=32.0,
               beta_slow=1.0, device=None):
    """(steps, amplitude): the table of turns per position of rotary_dim / 2 pairs, 64-bit fractions in an int64
    tensor on `device`, and the factor of the rotated pairs.  scaling: none, linear, ntk or yarn."""
    steps = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.int64)
    amplitude = _f()
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling is one of %s" % ", ".join(ROPE_SCALINGS))
    _check(lib.pa_rope_steps(steps.data_ptr() if steps.numel() else None, ctypes.byref(amplitude), rotary_dim, base,
                             ROPE_SCALINGS[scaling], factor, original_len, beta_fast, beta_slow), "pa_rope_steps")
    return (steps if device is None else steps.to(device)), amplitude.value


def _here(t):
    """The current device, which `t` has to be on."""
    d = t.get_device()
    if d < 0 or d != torch._C._cuda_getDevice():
        raise ValueError("tensors must be on the current CUDA device")
    return d


def _strided(t, n, dim, dtype, dev, what):
    """(pointer, token stride, head stride, heads) of a [n, heads, dim] view whose innermost stride is 1."""
    shape, s = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != n or shape[2] != dim or t.dtype is not dtype or (s[2] != 1 and dim > 1):
        raise ValueError("%s is [tokens, heads, head_dim] of one type, its elements next to each other" % what)
    if t.get_device() != dev:
        raise ValueError("tensors must be on the current CUDA device")
    h = shape[1]
    return t.data_ptr(), (s[0] if n > 1 else 0), (s[1] if h > 1 else 0), h


def _turn(x, out, n, dim, dtype, dev, what):
    """Checks and marshals a rotated tensor and where it goes: (out rows, x rows, heads)."""
    src = _strided(x, n, dim, dtype, dev, what)
    dst = src if out is None else _strided(out, n, dim, dtype, dev, what + "_out")
    p, s0, s1, h = dst
    if h != src[3]:
        raise ValueError("%s and %s_out have the same heads" % (what, what))
    # no element of the output lies in two places of it
    if n and h and not ((h == 1 or s1 >= dim) and (n == 1 or s0 >= s1 * (h - 1) + dim) or
                        (n == 1 or s0 >= dim) and (h == 1 or s1 >= s0 * (n - 1) + dim)):
        raise ValueError("the rows of %s overlap" % what)
    return p, s0, s1, src[0], src[1], src[2], h


_NO_TURN = (None, 0, 0, None, 0, 0, 0)


def _angles(positions, steps, n, dev):
    """(pointer of the positions, pointer of the steps, rotary_dim)"""
    if positions.dtype is not _I32 or positions.dim() != 1 or positions.numel() != n:
        raise TypeError("positions is int32 [tokens]")
    if steps.dtype is not torch.int64 or steps.dim() != 1:
        raise TypeError("steps is the int64 table of rope_steps")
    if positions.get_device() != dev or steps.get_device() != dev:
        raise ValueError("tensors must be on the current CUDA device")
    if not (positions.is_contiguous() and steps.is_contiguous()):
        raise ValueError("tensors must be contiguous")
    return positions.data_ptr(), steps.data_ptr(), 2 * steps.numel()


def _slots(slot_mapping, n, dev):
    if slot_mapping.dtype is not torch.int64 or slot_mapping.dim() != 1 or slot_mapping.numel() != n:
        raise TypeError("slot_mapping is int64 [tokens]")
    if slot_mapping.get_device() != dev or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be contiguous and on the current CUDA device")
    return slot_mapping.data_ptr()


def _float_kind(t):
    k = _KIND.get(t.dtype)
    if k is None or k == PA_FP8_E4M3:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return k


def _layout(layout):
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout is half or interleaved")
    return ROPE_LAYOUTS[layout]


def rope(q, k, positions, steps, amplitude=1.0, layout="half", q_out=None, k_out=None, stream=None):
    """Rotate the first 2 * len(steps) elements of every head of q [T, Hq, D] and k [T, Hkv, D] (either may be None;
    strided views will do) by the tokens' positions: in place, or into q_out / k_out.  Returns what it wrote."""
    x = q if q is not None else k
    if x is None or (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("q or k, and outputs for what is given")
    shape, dtype = x.shape, x.dtype
    if len(shape) != 3:
        raise ValueError("q and k are [tokens, heads, head_dim]")
    n, _, dim = shape
    kind, dev = _float_kind(x), _here(x)
    pos, table, rot = _angles(positions, steps, n, dev)
    qa = _NO_TURN if q is None else _turn(q, q_out, n, dim, dtype, dev, "q")
    ka = _NO_TURN if k is None else _turn(k, k_out, n, dim, dtype, dev, "k")
    _check(lib.pa_rope(*qa, *ka, pos, n, dim, rot, _layout(layout), table, amplitude, kind, _on(stream, dev)), "pa_rope")
    return (q if q_out is None else q_out), (k if k_out is None else k_out)


def rope_and_cache(q, key, value, positions, slot_mapping, k_cache, v_cache, steps, amplitude=1.0, layout="half",
                   q_out=None, stream=None):
    """Rotate q [T, Hq, D] (in place, or into q_out; None leaves it out) and append the rotated key and the value
    [T, Hkv, D] to the pool slots named by slot_mapping.  q, key and value may be strided views."""
    NB, bs, H, D, kind = _pools(k_cache, v_cache)
    if kind == PA_FP8_E4M3:
        raise TypeError("rotate first, then append to an e4m3 pool")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    n, dtype, dev = key.size(0), k_cache.dtype, _here(key)
    if k_cache.get_device() != dev or v_cache.get_device() != dev or not (
            k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the pools must be contiguous and on the current CUDA device")
    pos, table, rot = _angles(positions, steps, n, dev)
    qa = _NO_TURN if q is None else _turn(q, q_out, n, D, dtype, dev, "q")
    *ka, kh = _strided(key, n, D, dtype, dev, "key")
    *va, vh = _strided(value, n, D, dtype, dev, "value")
    if kh != H or vh != H:
        raise ValueError("key and value are [tokens, num_kv_heads, head_dim]")
    _check(lib.pa_rope_and_cache(*qa, *ka, *va, H, pos, _slots(slot_mapping, n, dev), n, k_cache.data_ptr(),
                                 v_cache.data_ptr(), NB, bs, D, rot, _layout(layout), table, amplitude, kind,
                                 _on(stream, dev)), "pa_rope_and_cache")
    return q if q_out is None else q_out


def _latent_pool(cache):
    shape = cache.shape
    if len(shape) != 3:
        raise ValueError("cache is [num_blocks, block_size, latent_dim + rope_dim]")
    return shape


def latent_append(latent, key_rope, positions, slot_mapping, cache, steps, amplitude=1.0, layout="half", query=None,
                  query_out=None, stream=None):
    """Append latent [T, R] and the rotated key_rope [T, P] to the slots of a latent cache [NB, bs, R + P]; query
    [T, H, P], the rotary part of the tokens' queries, is rotated along (in place, or into query_out).  Rows may be
    strided."""
    NB, bs, width = _latent_pool(cache)
    lshape, kshape, ls, ks = latent.shape, key_rope.shape, latent.stride(), key_rope.stride()
    n, dtype, kind, dev = lshape[0], cache.dtype, _float_kind(cache), _here(cache)
    if len(lshape) != 2 or len(kshape) != 2 or kshape[0] != n or latent.dtype is not dtype or (
            key_rope.dtype is not dtype) or ls[1] != 1 or ks[1] != 1:
        raise ValueError("latent and key_rope are [tokens, dim] of the cache's type, elements next to each other")
    if latent.get_device() != dev or key_rope.get_device() != dev or not cache.is_contiguous():
        raise ValueError("tensors must be on the current CUDA device, and the cache contiguous")
    if query is None and query_out is not None:
        raise ValueError("query_out without query")
    R, P = lshape[1], kshape[1]
    pos, table, rot = _angles(positions, steps, n, dev)
    if R + P != width or rot != P:
        raise ValueError("cache rows are latent_dim + rope_dim, and steps has rope_dim / 2 entries")
    qa = _NO_TURN if query is None else _turn(query, query_out, n, P, dtype, dev, "query")
    _check(lib.pa_latent_append(latent.data_ptr(), ls[0] if n > 1 else 0, key_rope.data_ptr(), ks[0] if n > 1 else 0,
                                *qa, pos, _slots(slot_mapping, n, dev), n, cache.data_ptr(), NB, bs, R, P,
                                _layout(layout), table, amplitude, kind, _on(stream, dev)), "pa_latent_append")
    return query if query_out is None else query_out


def alloc_latent_workspace(q, cache, block_tables):
    """Workspace for latent_decode with these sizes."""
    rows, H, width = q.shape
    R = (width - 16) // 128 * 128            # the one latent_dim of rows of this width
    n = lib.pa_latent_decode_workspace_bytes(rows, block_tables.shape[0], H, R)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)


def latent_decode(out, q, cache, block_tables, context_lens, scale, query_start=None, workspace=None, stream=None):
    """out[rows, H, R] = attention of q[rows, H, R + P] over a latent cache [NB, bs, R + P], whose rows' first R
    elements are the values too.  One row a sequence, or sequence b's rows are query_start[b]..query_start[b+1]-1,
    the last tokens of its context, causal."""
    NB, bs, width = _latent_pool(cache)
    B, cols = _table(block_tables, context_lens)
    qs, shape, dtype = q.shape, out.shape, cache.dtype
    if len(qs) != 3 or len(shape) != 3 or qs[2] != width or shape[0] != qs[0] or shape[1] != qs[1] or not (
            q.dtype is dtype and out.dtype is dtype):
        raise ValueError("q is [rows, num_heads, latent_dim + rope_dim], out [rows, num_heads, latent_dim], of the "
                         "cache's type")
    rows, H, R = shape
    kind = _float_kind(q)
    start = None
    if query_start is not None:
        _starts(query_start, B)
        _ready(query_start)
        start = query_start.data_ptr()
    elif rows != B:
        raise ValueError("one query row per sequence")
    if workspace is None:
        workspace = _own(alloc_latent_workspace, stream, q, cache, block_tables)
    dev = _ready(out, q, cache, block_tables, context_lens, workspace)
    _check(lib.pa_latent_decode(out.data_ptr(), q.data_ptr(), start, rows, cache.data_ptr(), block_tables.data_ptr(),
                                cols, context_lens.data_ptr(), B, H, R, width - R, bs, NB, scale,
                                workspace.data_ptr(), workspace.nbytes, kind, _on(stream, dev)), "pa_latent_decode")
    return out


def latent_prefill(out, q, query_start, kv, key_rope, kv_start, scale, stream=None):
    """Ragged causal attention over expanded latent vectors: q [rows, H, Dk + P], kv [T, H, Dk + Dv] (keys, then
    values, of every head), key_rope [T, P] shared by the heads (rows may be strided), out [rows, H, Dv].  Sequence
    b's context is rows kv_start[b]..kv_start[b+1]-1, its queries query_start[b]..query_start[b+1]-1, the last of it."""
    if not (q.dim() == kv.dim() == out.dim() == 3 and key_rope.dim() == 2) or not (
            q.dtype is kv.dtype and out.dtype is kv.dtype and key_rope.dtype is kv.dtype):
        raise ValueError("q, kv and out are [rows, num_heads, dim], key_rope [rows, rope_dim], of one type")
    rows, H, Dv = out.shape
    T, P = key_rope.shape
    Dk = q.size(2) - P
    if q.shape[:2] != out.shape[:2] or kv.shape != (T, H, Dk + Dv) or (key_rope.stride(1) != 1 and P > 1):
        raise ValueError("q is [rows, H, Dk + P], kv [T, H, Dk + Dv], key_rope [T, P], out [rows, H, Dv]")
    B = query_start.size(0) - 1
    _starts(query_start, B)
    _starts(kv_start, B)
    kind = _float_kind(q)
    dev = _ready(out, q, kv, query_start, kv_start)
    if key_rope.get_device() != dev:
        raise ValueError("tensors must be on the current CUDA device")
    _check(lib.pa_latent_prefill(out.data_ptr(), q.data_ptr(), query_start.data_ptr(), rows, kv.data_ptr(),
                                 key_rope.data_ptr(), key_rope.stride(0) if T > 1 else P, kv_start.data_ptr(), T, B, H, Dk, P,
                                 Dv, scale, kind, _on(stream, dev)), "pa_latent_prefill")
    return out


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
