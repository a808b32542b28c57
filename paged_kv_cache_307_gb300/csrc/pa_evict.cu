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
// select_kernel, one CTA or a cluster of four per (sequence, KV head): the keys (an
// order-preserving integer image of the weights, protected tokens above all
// others) are read once into shared memory, a quarter of the slots by each CTA of a
// cluster; the budget-th largest comes out by radix selection, 8 bits a pass, each
// pass with bins of its own, cleared at the start, the cluster's bins added up over
// distributed shared memory.  Each warp then owns a run of consecutive slots and
// walks it 32 at a time: a sweep that counts ties, one that decides what stays (ties
// by the lower slot; a bit per slot is kept), one that numbers the holes and the
// movers; between sweeps one scan over the warps and CTAs.  Weights, positions and
// the list of moves come out of it.
// Weights share their leading bits, and 32 lanes adding to one word take 32 turns: the
// first pass adds once per digit and warp, and the bins exist twice.
// move_kernel, one warp per destination block: the block's moves, a lane each,
// then their rows with eight 16-byte loads in flight per lane; over an e4m3 pool
// the block's scale becomes the largest of its own and the incoming rows' and the
// rows are requantised (the scales are powers of two: exact but for underflow).
// One warp owns a destination block's head, so nothing is atomic.
// Bound by latency and HBM: 8 bytes read per token and head, 8 written per slot,
// and the moved rows.  4 prompts of 4096 to 16384 tokens x 8 heads (bf16) cut to 2048
// take 37 us (45 with the cluster's bins added by one warp, a scan each for holes and
// movers, and ties counted in any case); a step of 64 sequences x 8 heads from at most
// 1040 tokens to 1024 (e4m3) 20.6 on the GPU.
#include <limits.h>

#include "pa_common.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_evict;

constexpr int kBins = 288;                // 256 digits, one word of padding after every 8
constexpr int kCopies = 2;
constexpr int kCluster = 4;
constexpr int kMaxSmemKeys = 48 * 1024;   // slots of a CTA whose keys fit in shared memory
constexpr int kMaxTokens = kCluster * 32 * kMaxSmemKeys;   // a bit for each slot in the room of the keys
constexpr int kMoveWarps = 8;

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

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int ld_cluster(const int* p, int rank) {
  uint32_t a;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// Every thread of the CTA, or of the cluster; what they wrote before is visible after.
template <int CS>
__device__ __forceinline__ void sync_all() {
  if constexpr (CS == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
}
// Exclusive sums of x and y (the same in every lane of a warp) over the warps of the
// cluster, and x's total.  buf [2][NW + 1] is used once.
template <int NW, int CS>
__device__ __forceinline__ void scan_warps(int& x, int& y, int (*buf)[NW + 1], int rank, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
    buf[0][warp] = x;
    buf[1][warp] = y;
  }
  __syncthreads();
  int sum[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int v = lane < NW ? buf[k][lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += u;
    }
    int before = __shfl_up_sync(0xffffffffu, v, 1);    // lane w: the warps before w
    if (lane == 0) before = 0;
    (k == 0 ? x : y) = __shfl_sync(0xffffffffu, before, warp);
    sum[k] = __shfl_sync(0xffffffffu, v, NW - 1);
  }
  total = sum[0];
  if constexpr (CS > 1) {
    if (threadIdx.x == 0) {
      buf[0][NW] = sum[0];
      buf[1][NW] = sum[1];
    }
    sync_all<CS>();
    total = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const int n0 = ld_cluster(&buf[0][NW], r), n1 = ld_cluster(&buf[1][NW], r);
      if (r < rank) {
        x += n0;
        y += n1;
      }
      total += n0;
    }
  }
}

// NT threads a CTA, CS CTAs a cluster.  SMEM: the keys are kept in shared memory
// (else recomputed from the inputs).  words: shared words for a CTA's stay bits.
template <int NT, int CS, bool SMEM>
__global__ void __launch_bounds__(NT) select_kernel(const EvictParams p, int words) {
  constexpr int NW = NT / 32;
  __shared__ int hist[4][kCopies][kBins];
  __shared__ int all[CS > 1 ? kBins : 1];
  __shared__ int wbuf[2][2][NW + 1];
  __shared__ int sh_digit, sh_left, sh_here;
  extern __shared__ uint32_t dyn[];
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = CS > 1 ? cluster_rank() : 0;
  const int bh = (int)blockIdx.x / CS, b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = rank * NT + tid;                   // thread of the cluster
  const int Lmax = p.max_blocks * p.bs;
  uint32_t* stay_bits = dyn;                         // this CTA's slots
  uint32_t* keys = dyn + words;                      // (SMEM)
  const int L0 = __ldg(&p.context_lens[b]);
  const int K0 = __ldg(&p.kept_lens[b]);
  const int seen = __ldg(&p.seen_lens[b]);
  for (int i = tid; i < 4 * kCopies * kBins; i += NT) (&hist[0][0][0])[i] = 0;
  const int L = clamp_len(L0, Lmax);
  const int kept = clamp_len(K0, L);
  const int newL = min(L, p.budget);
  if (h == 0 && gid == 0) {
    if (L0 != L || K0 != kept) atomicOr(&g_status_evict, PA_DEV_BAD_LEN);
    p.ws_len[b] = newL;
  }
  const size_t row = (size_t)bh * p.stride;
  const float* w = p.weights + row;
  const int32_t* tp = p.token_pos + row;
  float* wo = p.weights_out + row;
  int32_t* po = p.pos_out + row;
  auto pos_of = [&](int t) { return t < kept ? tp[t] : seen - L + t; };
  int32_t* first = p.first + (size_t)bh * (p.nb + 1);
  // the rest of the two rows: 0 and -1 from slot t on
  auto clear_from = [&](int t) {
#pragma unroll 4
    for (int x = t + gid; x < Lmax; x += CS * NT) {
      wo[x] = 0.f;
      po[x] = -1;
    }
  };
  if (L <= p.budget) {
    // nothing leaves (in and out may be the same rows: each thread reads its entry before writing it)
#pragma unroll 4
    for (int t = gid; t < L; t += CS * NT) {
      const float wt = w[t];
      const int pt = pos_of(t);
      wo[t] = wt;
      po[t] = pt;
    }
    clear_from(L);
    for (int j = gid; j <= p.nb; j += CS * NT) first[j] = 0;
    return;
  }
  // this CTA's slots: [base, base + n), a multiple of 32 but for the end
  const int per = CS > 1 ? (((L + CS - 1) / CS + 31) & ~31) : L;
  const int base = min(L, rank * per), n = min(L - base, per);
  auto make_key = [&](int t) -> uint32_t {
    const float wt = w[t];
    const int pos = pos_of(t);
    return pos < p.sinks || pos >= seen - p.recent ? 0xffffffffu : order_key(wt);
  };
  if constexpr (SMEM) {
#pragma unroll 8
    for (int i = tid; i < n; i += NT) keys[i] = make_key(base + i);
  }
  auto key_of = [&](int i) -> uint32_t {             // slot base + i
    if constexpr (SMEM) return keys[i];
    else return make_key(base + i);
  };
  __syncthreads();
  // ---- the budget-th largest key: 8 bits a pass from the top
  uint32_t prefix = 0, mask = 0;
  int left = p.budget;                    // how many of the keys that match the prefix are kept,
  int here = 0;                           // and how many match it
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* bins = hist[pass][lane & (kCopies - 1)];
    if (pass == 0) {
      // the leading bits of most weights are the same few: one addition per digit and warp
      for (int i0 = tid - lane; i0 < n; i0 += NT) {
        const bool in = i0 + lane < n;
        const int d = in ? (int)(key_of(i0 + lane) >> 24) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (in && (same & ((1u << lane) - 1u)) == 0) atomicAdd(&bins[d + (d >> 3)], __popc(same));
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < n; i += NT) {
        const uint32_t k = key_of(i);
        const int d = (int)(k >> shift) & 255;
        if ((k & mask) == prefix) atomicAdd(&bins[d + (d >> 3)], 1);
      }
    }
    sync_all<CS>();
    if constexpr (CS > 1) {
      // the cluster's bins, a digit per thread
      if (tid < 256) {
        int n = 0;
#pragma unroll
        for (int r = 0; r < CS; ++r)
#pragma unroll
          for (int k = 0; k < kCopies; ++k) n += ld_cluster(&hist[pass][k][tid + (tid >> 3)], r);
        all[tid + (tid >> 3)] = n;
      }
      __syncthreads();
    }
    if (warp == 0) {
      // lane l holds digits 255-8l .. 248-8l, the largest first: 9 (31 - l) + 7 - i in the padded bins
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = 9 * (31 - lane) + 7 - i;
        if constexpr (CS > 1) {
          c[i] = all[at];
        } else {
          c[i] = 0;
#pragma unroll
          for (int k = 0; k < kCopies; ++k) c[i] += hist[pass][k][at];
        }
        sum += c[i];
      }
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      int before = incl - sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < left && left <= before + c[i]) {     // in exactly one lane
          sh_digit = 255 - 8 * lane - i;
          sh_left = left - before;
          sh_here = c[i];
        }
        before += c[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sh_digit << shift;
    left = sh_left;
    here = sh_here;
    mask |= 0xffu << shift;
    // (the next write to the pair comes after a barrier)
  }
  // keys above `prefix` are kept, and the first `left` of those equal to it

  // ---- each warp's run of slots, 32 at a time
  const int run = ((n + NT - 1) / NT) * 32;
  const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
  const unsigned lt = (1u << lane) - 1u;
  // ties before the run (where all that tie are kept, their order is no matter)
  int ties = 0, total;
  if (here != left) {
    for (int i0 = r0; i0 < r1; i0 += 32)
      ties += __popc(__ballot_sync(0xffffffffu, i0 + lane < r1 && key_of(i0 + lane) == prefix));
    int none = 0;
    scan_warps<NW, CS>(ties, none, wbuf[0], rank, total);
  } else {
    left = INT_MAX;
  }
  // slots of the 32 from base + i0 that are in the run, and those below the budget
  auto in_run = [&](int i0) -> unsigned { return r1 - i0 >= 32 ? 0xffffffffu : (1u << (r1 - i0)) - 1u; };
  auto below = [&](int i0) -> unsigned {
    const int t0 = base + i0;
    return t0 + 32 <= p.budget ? 0xffffffffu : t0 < p.budget ? (1u << (p.budget - t0)) - 1u : 0u;
  };
  int holes = 0, movers = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const bool in = i0 + lane < r1;
    const uint32_t k = in ? key_of(i0 + lane) : 0u;
    const unsigned me = __ballot_sync(0xffffffffu, in && k == prefix);
    const unsigned s =
        __ballot_sync(0xffffffffu, in && (k > prefix || (k == prefix && ties + __popc(me & lt) < left)));
    ties += __popc(me);
    if (lane == 0) stay_bits[i0 >> 5] = s;
    holes += __popc(in_run(i0) & below(i0) & ~s);
    movers += __popc(s & ~below(i0));
  }
  int hole0 = holes, mover0 = movers;
  scan_warps<NW, CS>(hole0, mover0, wbuf[1], rank, total);
  const int nmove = total;                             // as many movers as holes
  Move* mv = p.moves + (size_t)bh * p.cap;
  int32_t* dst = p.dst + (size_t)bh * p.cap;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const unsigned s = stay_bits[i0 >> 5], low = in_run(i0) & below(i0);
    const unsigned hm = low & ~s, cm = s & ~below(i0), bit = 1u << lane;
    const int t = base + i0 + lane;
    if (low & bit) {
      const int at = hole0 + __popc(hm & lt);
      if ((t & (p.bs - 1)) == 0) first[t / p.bs] = at;
      if (hm & bit) dst[at] = t;
    } else if (cm & bit) {
      mv[mover0 + __popc(cm & lt)].src = t;
    }
    hole0 += __popc(hm);
    mover0 += __popc(cm);
  }
  if (gid == 0) first[p.nb] = nmove;
  sync_all<CS>();
  // ---- what stays below the budget, the movers' weights, positions and scales, then the rest of the
  // rows (in and out may be the same: a slot below the budget is read by its own thread only, and the
  // movers' slots are cleared after they have been read)
#pragma unroll 4
  for (int i = tid; i < min(n, newL - base); i += NT) {
    if ((stay_bits[i >> 5] >> (i & 31)) & 1u) {
      const int t = base + i;
      const float wt = w[t];
      const int pt = pos_of(t);
      wo[t] = wt;
      po[t] = pt;
    }
  }
#pragma unroll 2
  for (int i = gid; i < nmove; i += CS * NT) {
    const int s = mv[i].src, d = dst[i];
    const float wt = w[s];
    const int pt = pos_of(s);
    if (p.elem == 1) {
      const int blk = __ldg(&p.block_tables[(size_t)b * p.max_blocks + s / p.bs]);
      if ((unsigned)blk < (unsigned)p.num_blocks) {
        mv[i].k_scale = p.scale[0][(size_t)blk * p.scale_row + h];
        mv[i].v_scale = p.scale[1][(size_t)blk * p.scale_row + h];
      }
    }
    wo[d] = wt;
    po[d] = pt;
  }
  sync_all<CS>();
  clear_from(newL);
}

// Two conversions of two values each, the first value in the low byte.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
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

// One CTA per (sequence, KV head) and `per` destination blocks.
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const EvictParams p, int per) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (p.nb + per - 1) / per;
  const int bh = (int)(blockIdx.x / groups), g0 = (int)(blockIdx.x % groups) * per;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int newL = p.ws_len[b];
  if (g0 == 0 && h == 0 && threadIdx.x == 0) p.new_lens[b] = newL;
  const int32_t* tab = p.block_tables + (size_t)b * p.max_blocks;
  const Move* mv = p.moves + (size_t)bh * p.cap;
  const int32_t* dst = p.dst + (size_t)bh * p.cap;
  const int rb = p.D * p.elem;                            // one head's row in bytes: 32 to 512
  const int csh = 31 - __clz(rb / 16), cpr = 1 << csh;    // its 16-byte chunks, a power of two
  const size_t tok = (size_t)p.Hkv * rb;                  // from token to token
  for (int j = g0 + warp; j < min(p.nb, g0 + per); j += kMoveWarps) {
    const int32_t* first = p.first + (size_t)bh * (p.nb + 1) + j;
    const int m0 = first[0], n = first[1] - m0;           // at most bs moves
    if (n <= 0) continue;
    const int dblk = __ldg(&tab[j]);
    if ((unsigned)dblk >= (unsigned)p.num_blocks) {
      if (lane == 0) atomicOr(&g_status_evict, PA_DEV_BAD_BLOCK);
      continue;
    }
    // lane i: move i
    long long srow = -1;                                  // source row in the pool, -1: its block is not one
    int drow = 0;
    float sc[2] = {0.f, 0.f};
    if (lane < n) {
      const Move m = mv[m0 + lane];
      const int sblk = __ldg(&tab[m.src / p.bs]);
      drow = dst[m0 + lane] - j * p.bs;
      sc[0] = m.k_scale;
      sc[1] = m.v_scale;
      if ((unsigned)sblk < (unsigned)p.num_blocks) srow = (long long)sblk * p.bs + m.src % p.bs;
      else atomicOr(&g_status_evict, PA_DEV_BAD_BLOCK);
    }
    float s[2] = {0.f, 0.f};
    if (p.elem == 1) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float* sp = p.scale[kv] + (size_t)dblk * p.scale_row + h;
        const float old = *sp;
        float x = srow >= 0 ? sc[kv] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
        s[kv] = fmaxf(old, x);
        __syncwarp();
        if (s[kv] > old) {
          if (lane == 0) *sp = s[kv];
          // the rows that stay in the block (the holes are overwritten below)
          unsigned char* dbase =
              static_cast<unsigned char*>(p.pool[kv]) + ((size_t)dblk * p.bs) * tok + (size_t)h * rb;
          const float f = old / s[kv];
          const int rows = min(p.bs, newL - j * p.bs);
          for (int c = lane; c < rows << csh; c += 32) {
            unsigned char* at = dbase + (size_t)(c >> csh) * tok + (size_t)(c & (cpr - 1)) * 16;
            *reinterpret_cast<uint4*>(at) = rescale16(*reinterpret_cast<const uint4*>(at), f);
          }
          __syncwarp();
        }
      }
    }
    // rows of K and V, four 16-byte chunks of each in flight per lane
    const unsigned char* kp = static_cast<const unsigned char*>(p.pool[0]) + (size_t)h * rb;
    const unsigned char* vp = static_cast<const unsigned char*>(p.pool[1]) + (size_t)h * rb;
    const size_t dbase = (size_t)dblk * p.bs;
    for (int c0 = 0; c0 < n << csh; c0 += 128) {
      uint4 x[4], y[4];
      long long sr[4];
      int dr[4];
      float sk[4], sv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 32 * k + lane, i = min(c >> csh, 31);
        sr[k] = __shfl_sync(0xffffffffu, srow, i);
        dr[k] = __shfl_sync(0xffffffffu, drow, i);
        sk[k] = __shfl_sync(0xffffffffu, sc[0], i);
        sv[k] = __shfl_sync(0xffffffffu, sc[1], i);
        if (c >= n << csh) sr[k] = -1;
        if (sr[k] >= 0) {
          const size_t at = (size_t)sr[k] * tok + (size_t)(c & (cpr - 1)) * 16;
          x[k] = *reinterpret_cast<const uint4*>(kp + at);
          y[k] = *reinterpret_cast<const uint4*>(vp + at);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (sr[k] < 0) continue;
        const int c = c0 + 32 * k + lane;
        const size_t at = (dbase + dr[k]) * tok + (size_t)h * rb + (size_t)(c & (cpr - 1)) * 16;
        if (p.elem == 1) {
          if (sk[k] != s[0]) x[k] = rescale16(x[k], s[0] > 0.f ? sk[k] / s[0] : 0.f);
          if (sv[k] != s[1]) y[k] = rescale16(y[k], s[1] > 0.f ? sv[k] / s[1] : 0.f);
        }
        st_v4(static_cast<unsigned char*>(p.pool[0]) + at, x[k]);
        st_v4(static_cast<unsigned char*>(p.pool[1]) + at, y[k]);
      }
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

unsigned* status_word_evict() { return device_word(g_status_evict); }

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
      !supported_head_dim(head_dim) || !supported_block_size(block_size) || max_ctx > kMaxTokens ||
      row_stride < max_ctx || budget <= 0 || recent < 0 || sinks < 0 || (long long)recent + sinks > budget ||
      (long long)num_seqs * num_kv_heads * kCluster > 0x7fffffffll)
    return PA_ERR_SHAPE;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !kept_lens || !seen_lens || !weights || !token_pos ||
      !new_lens || !weights_out || !token_pos_out || (fp8 && (!k_scale || !v_scale)))
    return PA_ERR_NULL;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace)) return PA_ERR_ALIGN;
  const Layout l = layout(num_seqs, num_kv_heads, max_blocks_per_seq, block_size, budget);
  if (!workspace || workspace_bytes < l.total) return PA_ERR_WORKSPACE;
  // destination blocks per CTA of the second kernel: a warp has one while the
  // (sequence, head) rows alone do not fill the SMs, four otherwise (32 rows 37 us
  // against 48 with four, 512 rows 28 with one against 22.5)
  const int rows = num_seqs * num_kv_heads, sms = device_sm_count();
  const int per = rows >= 2 * sms ? 4 * kMoveWarps : kMoveWarps;
  const long long blocks = (long long)rows * ((l.nb + per - 1) / per);
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
  // A row of up to 2048 slots has one CTA of 256 threads (512 rows of 1040 slots: 22 us; clusters 93).  A
  // longer one has 512 (32 rows of 4000 slots 21 us against 26, 512 rows 97 against 91; 128 rows of 16384
  // 65 against 86), or a cluster of four of them while the rows leave SMs idle (64 rows of 16384 slots 36 us
  // against 46, 32 of 6000 22 against 24; but 128 of 16384 73 against 65) and where a CTA's shared memory
  // does not hold the keys.
  const bool tall = max_ctx > 2048, wide = tall && (rows * kCluster <= 2 * sms || max_ctx > kMaxSmemKeys);
  const int cs = wide ? kCluster : 1;
  const long long slots = wide ? ((max_ctx + cs - 1) / cs + 31) / 32 * 32 : max_ctx;    // of a CTA
  const bool in_smem = slots <= kMaxSmemKeys;
  int words = (int)((slots + 31) / 32);
  const size_t smem = (size_t)words * 4 + (in_smem ? (size_t)slots * 4 : 0);
  const void* select = !tall     ? reinterpret_cast<const void*>(&select_kernel<256, 1, true>)
                       : !wide   ? reinterpret_cast<const void*>(&select_kernel<512, 1, true>)
                       : in_smem ? reinterpret_cast<const void*>(&select_kernel<512, kCluster, true>)
                                 : reinterpret_cast<const void*>(&select_kernel<512, kCluster, false>);
  if (smem > 32 * 1024) {
    // (static bins of 9 KB come on top)
    if (!ck(cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, 204 * 1024),
            "cudaFuncSetAttribute(select_kernel)"))
      return PA_ERR_CUDA;
  }
  void* args[] = {&p, &words};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cs));
  cfg.blockDim = dim3(tall ? 512u : 256u);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cs;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = wide ? 1 : 0;
  if (!ck(cudaLaunchKernelExC(&cfg, select, args), "cudaLaunchKernelExC(select_kernel)")) return PA_ERR_CUDA;
  int per_arg = per;
  void* margs[] = {&p, &per_arg};
  if (!ck(launch_after(reinterpret_cast<const void*>(&move_kernel), dim3((unsigned)blocks), dim3(kMoveWarps * 32),
                       margs, (cudaStream_t)stream),
          "cudaLaunchKernel(move_kernel)"))
    return PA_ERR_CUDA;
  return PA_OK;
}
