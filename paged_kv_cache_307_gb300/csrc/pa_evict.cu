// pa_evict.cu — cut the cache of every (sequence, KV head) to a budget of
// tokens, keeping those with the largest accumulated attention weight.
//
// Softmax attention is a sum over tokens, so the order of a cache's rows does
// not matter to it.  What stays below the budget therefore stays where it is,
// and the i-th kept row at or above the budget moves into the i-th slot below it
// whose token was dropped: as many rows move as slots were freed, sources and
// destinations are disjoint sets, and no move waits for another.  (Closing the
// gaps in order would move almost every row behind the first gap, and in
// sequence.)  A token's position in the text then no longer follows from its
// slot, so it is carried in token_pos.
//
// select_kernel, one CTA per (sequence, KV head): the budget-th largest key by
// radix selection, 8 bits a pass over an order-preserving integer image of the
// weights (protected tokens above all others); then one pass in slot order
// that marks what is kept, breaking ties by the lower slot, and numbers the
// holes and the movers by a block-wide scan; weights, positions and the list
// of moves come out of it.
// move_kernel, one warp per (sequence, KV head, destination block): its rows
// are copied in; over an e4m3 pool the block's scale becomes the largest of
// its own and the incoming rows' and the rows are requantised (the scales are
// powers of two: exact but for underflow).  One warp owns a destination
// block's head, so nothing is atomic.
// Bound by latency and HBM: 8 bytes read per token and head, 8 written per slot,
// and the moved rows.
#include "pa_common.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_evict;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveWarps = 4;

struct Move {
  int32_t src;          // slot the row comes from
  float k_scale, v_scale;  // e4m3 pools: that block's scales before the call
};

struct EvictParams {
  void* pool[2];
  float* scale[2];
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* kept_lens;
  const int32_t* seen_lens;
  const float* weights;
  const int32_t* token_pos;
  int32_t* new_lens;
  float* weights_out;
  int32_t* pos_out;
  long long stride;        // floats (ints) per (sequence, head) row of the four tables
  int B, Hkv, D, bs, max_blocks, num_blocks, scale_row, elem;
  int budget, recent, sinks;
  int nb;                  // destination blocks per sequence: ceil(min(budget, max_blocks * bs) / bs)
  int cap;                 // moves per (sequence, head) at most
  Move* moves;             // [B * Hkv][cap]
  int32_t* dst;            // [B * Hkv][cap] destination slots, ascending
  int32_t* first;          // [B * Hkv][nb + 1] first move into each destination block
  int32_t* ws_len;         // [B] new lengths
};

// Larger key = kept first.  NaN ranks with the lowest weights.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w == w ? w + 0.f : -INFINITY);     // -0 counts as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int clamp_len(int L, int Lmax) { return L < 0 ? 0 : min(L, Lmax); }

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int wsum[2][kSelWarps];
  __shared__ int sh_digit, sh_left;
  const int bh = (int)blockIdx.x, b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Lmax = p.max_blocks * p.bs;
  const int L0 = __ldg(&p.context_lens[b]);
  const int L = clamp_len(L0, Lmax);
  const int K0 = __ldg(&p.kept_lens[b]);
  const int kept = clamp_len(K0, L);
  const int seen = __ldg(&p.seen_lens[b]);
  if (h == 0 && tid == 0) {
    if (L0 != L || K0 != kept) atomicOr(&g_status_evict, PA_DEV_BAD_LEN);
    p.ws_len[b] = min(L, p.budget);
  }
  const size_t row = (size_t)bh * p.stride;
  const float* w = p.weights + row;
  const int32_t* tp = p.token_pos + row;
  float* wo = p.weights_out + row;
  int32_t* po = p.pos_out + row;
  const int newL = min(L, p.budget);
  auto pos_of = [&](int t) { return t < kept ? tp[t] : seen - L + t; };
  auto key_of = [&](int t) -> uint32_t {
    const int pos = pos_of(t);
    return pos < p.sinks || pos >= seen - p.recent ? 0xffffffffu : order_key(w[t]);
  };
  int32_t* first = p.first + (size_t)bh * (p.nb + 1);
  if (L <= p.budget) {
    // nothing leaves (in and out may be the same rows: each thread reads its entry before writing it)
    for (int t = tid; t < Lmax; t += kSelThreads) {
      const float wt = t < L ? w[t] : 0.f;
      const int pt = t < L ? pos_of(t) : -1;
      wo[t] = wt;
      po[t] = pt;
    }
    for (int j = tid; j <= p.nb; j += kSelThreads) first[j] = 0;
    return;
  }
  // ---- the budget-th largest key: 8 bits a pass from the top
  uint32_t prefix = 0, mask = 0;
  int left = p.budget;                    // how many of the keys that match the prefix are kept
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int t = tid; t < L; t += kSelThreads) {
      const uint32_t k = key_of(t);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255-8l .. 248-8l, the largest first
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = hist[255 - 8 * lane - i];
        sum += c[i];
      }
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      int before = incl - sum;
      if (before < left && left <= incl) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < left && left <= before + c[i]) {
            sh_digit = 255 - 8 * lane - i;
            sh_left = left - before;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh_digit << shift;
    mask |= 0xffu << shift;
    left = sh_left;
    __syncthreads();
  }
  // keys above `prefix` are kept, and the first `left` of those equal to it

  // ---- one pass in slot order: kept, holes below the budget, movers at or above it
  Move* mv = p.moves + (size_t)bh * p.cap;
  int32_t* dst = p.dst + (size_t)bh * p.cap;
  int ties = 0, holes = 0, movers = 0;    // running counts over the slots before this tile
  for (int t0 = 0; t0 < L; t0 += kSelThreads) {
    const int t = t0 + tid;
    const uint32_t k = t < L ? key_of(t) : 0u;
    const bool eq = t < L && k == prefix;
    const unsigned lt = (1u << lane) - 1u;
    const unsigned me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) wsum[0][warp] = __popc(me);
    __syncthreads();
    int eb = ties, et = 0;
    for (int i = 0; i < kSelWarps; ++i) {
      if (i < warp) eb += wsum[0][i];
      et += wsum[0][i];
    }
    const bool stay = t < L && (k > prefix || (eq && eb + __popc(me & lt) < left));
    const bool hole = t < p.budget && !stay, come = t >= p.budget && stay;
    const unsigned mh = __ballot_sync(0xffffffffu, hole || come);
    // a tile may hold both kinds: holes below the budget, movers from it on
    const unsigned mhole = __ballot_sync(0xffffffffu, hole);
    if (lane == 0) wsum[1][warp] = __popc(mhole) | (__popc(mh & ~mhole) << 16);
    __syncthreads();
    int hb = holes, cb = movers, ht = 0, ct = 0;
    for (int i = 0; i < kSelWarps; ++i) {
      const int v = wsum[1][i];
      if (i < warp) {
        hb += v & 0xffff;
        cb += v >> 16;
      }
      ht += v & 0xffff;
      ct += v >> 16;
    }
    hb += __popc(mhole & lt);
    cb += __popc(mh & ~mhole & lt);
    if (t < p.budget) {
      if ((t % p.bs) == 0) first[t / p.bs] = hb;
      if (hole) dst[hb] = t;
      else {
        // (in and out may be the same row)
        const float wt = w[t];
        const int pt = pos_of(t);
        wo[t] = wt;
        po[t] = pt;
      }
    } else if (come) {
      Move m;
      m.src = t;
      m.k_scale = m.v_scale = 0.f;
      mv[cb] = m;
    }
    ties += et;
    holes += ht;
    movers += ct;
    __syncthreads();
  }
  if (tid == 0) first[p.nb] = holes;
  __syncthreads();
  // ---- the movers' weights, positions and scales, then the rest of the rows
  for (int i = tid; i < holes; i += kSelThreads) {
    const int s = mv[i].src;
    wo[dst[i]] = w[s];
    po[dst[i]] = pos_of(s);
    if (p.elem == 1) {
      const int blk = __ldg(&p.block_tables[(size_t)b * p.max_blocks + s / p.bs]);
      if ((unsigned)blk < (unsigned)p.num_blocks) {
        mv[i].k_scale = p.scale[0][(size_t)blk * p.scale_row + h];
        mv[i].v_scale = p.scale[1][(size_t)blk * p.scale_row + h];
      }
    }
  }
  __syncthreads();
  for (int t = newL + tid; t < Lmax; t += kSelThreads) {
    wo[t] = 0.f;
    po[t] = -1;
  }
}

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float_to_fp8(b, __NV_SATFINITE, __NV_E4M3) << 8 |
         (uint32_t)__nv_cvt_float_to_fp8(c, __NV_SATFINITE, __NV_E4M3) << 16 |
         (uint32_t)__nv_cvt_float_to_fp8(d, __NV_SATFINITE, __NV_E4M3) << 24;
}
// Sixteen codes times f.
__device__ __forceinline__ uint4 rescale16(uint4 x, float f) {
  float v[16];
  Elem<fp8e4m3>::unpack(x, v);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] *= f;
  return make_uint4(encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7]),
                    encode4(v[8], v[9], v[10], v[11]), encode4(v[12], v[13], v[14], v[15]));
}

__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const EvictParams p) {
  const int lane = threadIdx.x & 31;
  const long long u = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  if (u >= (long long)p.B * p.Hkv * p.nb) return;
  const int j = (int)(u % p.nb);
  const int bh = (int)(u / p.nb), b = bh / p.Hkv, h = bh % p.Hkv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int newL = p.ws_len[b];
  if (j == 0 && h == 0 && lane == 0) p.new_lens[b] = newL;
  const int32_t* first = p.first + (size_t)bh * (p.nb + 1) + j;
  const int m0 = first[0], m1 = first[1];
  if (m0 >= m1) return;
  const int32_t* tab = p.block_tables + (size_t)b * p.max_blocks;
  const int dblk = __ldg(&tab[j]);
  if ((unsigned)dblk >= (unsigned)p.num_blocks) {
    if (lane == 0) atomicOr(&g_status_evict, PA_DEV_BAD_BLOCK);
    return;
  }
  const Move* mv = p.moves + (size_t)bh * p.cap;
  const int32_t* dst = p.dst + (size_t)bh * p.cap;
  const int rb = p.D * p.elem, cpr = rb / 16;             // one head's row, in 16-byte chunks
  const size_t tok = (size_t)p.Hkv * rb;                  // from token to token
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    unsigned char* pool = static_cast<unsigned char*>(p.pool[kv]);
    unsigned char* dbase = pool + ((size_t)dblk * p.bs) * tok + (size_t)h * rb;
    float s = 0.f, old = 0.f;
    if (p.elem == 1) {
      float* sp = p.scale[kv] + (size_t)dblk * p.scale_row + h;
      old = *sp;
      s = old;
      for (int i = m0 + lane; i < m1; i += 32) s = fmaxf(s, kv ? mv[i].v_scale : mv[i].k_scale);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, off));
      __syncwarp();
      if (s > old) {
        if (lane == 0) *sp = s;
        // the rows that stay in the block (the holes are overwritten below)
        const float f = old / s;
        const int rows = min(p.bs, newL - j * p.bs);
        for (int c = lane; c < rows * cpr; c += 32) {
          unsigned char* at = dbase + (size_t)(c / cpr) * tok + (size_t)(c % cpr) * 16;
          *reinterpret_cast<uint4*>(at) = rescale16(*reinterpret_cast<const uint4*>(at), f);
        }
        __syncwarp();
      }
    }
    for (int c = lane; c < (m1 - m0) * cpr; c += 32) {
      const int i = m0 + c / cpr;
      const Move m = mv[i];
      const int sblk = __ldg(&tab[m.src / p.bs]);
      if ((unsigned)sblk >= (unsigned)p.num_blocks) {
        atomicOr(&g_status_evict, PA_DEV_BAD_BLOCK);
        continue;
      }
      const unsigned char* from =
          pool + ((size_t)sblk * p.bs + m.src % p.bs) * tok + (size_t)h * rb + (size_t)(c % cpr) * 16;
      unsigned char* to = dbase + (size_t)(dst[i] - j * p.bs) * tok + (size_t)(c % cpr) * 16;
      uint4 x = *reinterpret_cast<const uint4*>(from);
      if (p.elem == 1) {
        const float ss = kv ? m.v_scale : m.k_scale;
        if (ss != s) x = rescale16(x, s > 0.f ? ss / s : 0.f);
      }
      st_v4(to, x);
    }
  }
}

struct Layout {
  size_t moves, dst, first, len, total;
  int nb, cap;
};
Layout layout(int B, int Hkv, int max_blocks, int bs, int budget) {
  Layout l;
  const long long max_ctx = (long long)max_blocks * bs;
  const long long keep = budget < max_ctx ? budget : max_ctx;
  l.nb = (int)((keep + bs - 1) / bs);
  long long cap = max_ctx - keep;               // rows move into freed slots from at or above the budget
  if (cap > keep) cap = keep;
  l.cap = (int)cap;
  const size_t rows = (size_t)B * Hkv;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.moves = 0;
  l.dst = up(rows * cap * sizeof(Move));
  l.first = l.dst + up(rows * cap * 4);
  l.len = l.first + up(rows * (l.nb + 1) * 4);
  l.total = l.len + up((size_t)B * 4);
  return l;
}

}  // namespace

unsigned fetch_status_evict() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_evict, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v && cudaMemcpyToSymbol(g_status_evict, &zero, sizeof(zero)) != cudaSuccess) return 0xffffffffu;
  return v;
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_evict_workspace_bytes(int num_seqs, int num_kv_heads, int max_blocks_per_seq, int block_size,
                                           int budget) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || !supported_block_size(block_size) ||
      budget <= 0)
    return 0;
  return layout(num_seqs, num_kv_heads, max_blocks_per_seq, block_size, budget).total;
}

extern "C" int pa_evict(void* k_cache, void* v_cache, float* k_scale, float* v_scale, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, const int32_t* kept_lens,
                        const int32_t* seen_lens, int num_seqs, const float* weights, const int32_t* token_pos,
                        int budget, int recent, int sinks, int32_t* new_lens, float* weights_out,
                        int32_t* token_pos_out, long long row_stride, int num_blocks, int block_size,
                        int num_kv_heads, int head_dim, void* workspace, size_t workspace_bytes, pa_dtype kv_dtype,
                        void* stream) {
  if (kv_dtype != PA_F32 && kv_dtype != PA_BF16 && kv_dtype != PA_FP8_E4M3) return PA_ERR_DTYPE;
  const bool fp8 = kv_dtype == PA_FP8_E4M3;
  const long long max_ctx = (long long)max_blocks_per_seq * block_size;
  if (num_seqs < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || num_kv_heads <= 0 ||
      !supported_head_dim(head_dim) || !supported_block_size(block_size) || max_ctx > 0x7fffffffll ||
      row_stride < max_ctx || budget <= 0 || recent < 0 || sinks < 0 || (long long)recent + sinks > budget ||
      (long long)num_seqs * num_kv_heads > 0x7fffffffll)
    return PA_ERR_SHAPE;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !kept_lens || !seen_lens || !weights || !token_pos ||
      !new_lens || !weights_out || !token_pos_out || (fp8 && (!k_scale || !v_scale)))
    return PA_ERR_NULL;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace)) return PA_ERR_ALIGN;
  const Layout l = layout(num_seqs, num_kv_heads, max_blocks_per_seq, block_size, budget);
  if (!workspace || workspace_bytes < l.total) return PA_ERR_WORKSPACE;
  const long long units = (long long)num_seqs * num_kv_heads * l.nb;
  const long long blocks = (units + kMoveWarps - 1) / kMoveWarps;
  if (blocks > 0x7fffffffll) return PA_ERR_SHAPE;
  EvictParams p;
  p.pool[0] = k_cache;
  p.pool[1] = v_cache;
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.kept_lens = kept_lens;
  p.seen_lens = seen_lens;
  p.weights = weights;
  p.token_pos = token_pos;
  p.new_lens = new_lens;
  p.weights_out = weights_out;
  p.pos_out = token_pos_out;
  p.stride = row_stride;
  p.B = num_seqs;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  p.bs = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.scale_row = scale_row(num_kv_heads);
  p.elem = elem_bytes(kv_dtype);
  p.budget = budget;
  p.recent = recent;
  p.sinks = sinks;
  p.nb = l.nb;
  p.cap = l.cap;
  char* ws = static_cast<char*>(workspace);
  p.moves = reinterpret_cast<Move*>(ws + l.moves);
  p.dst = reinterpret_cast<int32_t*>(ws + l.dst);
  p.first = reinterpret_cast<int32_t*>(ws + l.first);
  p.ws_len = reinterpret_cast<int32_t*>(ws + l.len);
  void* args[] = {&p};
  if (!ck(cudaLaunchKernel(reinterpret_cast<const void*>(&select_kernel), dim3((unsigned)(num_seqs * num_kv_heads)),
                           dim3(kSelThreads), args, 0, (cudaStream_t)stream),
          "cudaLaunchKernel(select_kernel)"))
    return PA_ERR_CUDA;
  if (!ck(launch_after(reinterpret_cast<const void*>(&move_kernel), dim3((unsigned)blocks), dim3(kMoveWarps * 32),
                       args, (cudaStream_t)stream),
          "cudaLaunchKernel(move_kernel)"))
    return PA_ERR_CUDA;
  return PA_OK;
}
