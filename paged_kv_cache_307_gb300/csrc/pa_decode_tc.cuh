// pa_decode_tc.cuh — paged decode attention over an e4m3 pool with one scale
// per (block, KV head) on the 5th-generation tensor cores (tcgen05.mma
// kind::f8f6f4): the codes go from HBM to shared memory by TMA and from there
// into the products as they are.  Shared by the translation units that
// instantiate it (pa_decode_fp8_blocks.cu, pa_decode_weights_fp8.cu).
//
// What bounds decode over 8-bit pools is not the bytes but the instructions
// that widen every code for 16-bit products (about 36 per token and KV head on
// the mma.sync path: 281 us where this takes 192).  Here a tile of 128 tokens of
// one KV head costs eight MMAs, and per token only its scores are touched by threads.
// Bound by HBM but for the CTAs' starts and ends: 64 requests x 8 KV heads x 128,
// 32 query heads, over U[1024, 16384] tokens take 192 us (1.14 GB, 6.0 TB/s, 88 % of
// the copy rate) and 64 x 32 heads over U[128, 2048] 96 us (6.0 TB/s).  P's third term
// costs nothing that shows there (193 and 94 us with two terms): the tensor pipe is idle
// enough, and threads store three bytes for two.  Where the threads' work bounds the
// call it is 1 %: 64 x 8 heads over U[1024, 8192] in groups of 8 121 us (120).
//
// One CTA = (sequence, partition of P tokens, KV head, up to 16 query heads):
//   S^T[128 tokens x N] = K[128 x 128] Q^T      A = K tile (K-major), B = Q rows
//   O^T[128 dims x N]  += V^T[128 x 128] P^T    A = V tile (MN-major), B = P rows
// N: every query head has several rows, because bf16 Q (8 significant bits) and P
// do not fit one 8-bit value.  Q has two e4m3 terms (N = 2 x 8 or 16):
//   q 2^-e = hi + lo / 16, hi = e4m3(q 2^-e), lo = e4m3(16 (q 2^-e - hi)),
// with 2^e per head so that max |q 2^-e| is in [128, 256).  The residual of hi
// has at most 4 significant bits left, so the split is exact while
// |q 2^-e| >= 2^-6, and off by at most 2^-14 (2^-21 of the largest) below.
// P has three e5m2 terms (N = 3 x 4, 8 or 16, rounded up to 16, 32, 48; the two
// operands' formats are independent):
//   x = 2^(z - w + 12) = t0 + t1 / 16 + t2 / 256, each term the rest's e5m2 value,
// z = score + log2 of its block's V scale, w the head's running reference for z,
// x <= 2^15.  Each term takes 3 bits, so x is held to 2^-9 of itself down to 2^-26 of
// the reference and to 2^-35 of the reference below: bf16's precision, and next to
// nothing lost of the many tokens of small weight that stand beside one that takes
// nearly all of it (two e4m3 terms dropped what is below 2^-19 of the reference, which
// was all of the output where the one had a value of zero), however far the blocks' scales are
// apart.  The sum of the softmax has a reference m of its own (a block may have the
// scale 0); the K scale multiplies the score in fp32.
//
// head_dim 64 and 32 (HP = 2 and 4): HP neighbouring KV heads make one row of 128
// codes, so the pool is read as one of Hkv / HP heads of 128.  The query heads of
// all of them share the CTA; a query row is zero outside its own KV head's
// columns, and of its output row only those are kept.  The products are HP times
// what they need be, and the tensor cores are idle enough for it.
//
//  * warp 4 (TMA): block-table entries and scales by parallel lanes, K and V
//    boxes {128 B, 1 head, bs rows} into 2-stage rings of 16 KB tiles; K's
//    stage frees with its S, V's with its O.  The first two tiles are requested
//    before the CTA's barrier, as soon as the length and their ids are there (by
//    the loop, behind their scales, the first request left 2000 clocks later: 196 us).
//  * warp 5: TMEM, and the MMAs: S_{j+1} before O += V_j P_j.
//  * warps 0-3: one thread per token: scores from TMEM, scale, mask, p = 2^(s-m),
//    the sum, P's three terms as bytes into the B tile.  The references (m and w of
//    every head) are common to the 128 threads and move only when a score or a z
//    exceeds its own by 3 (a factor 8): one barrier with a vote per tile; then O is
//    rescaled in TMEM.
//  * 74 KB of shared memory for up to 8 heads: three CTAs per SM, so one CTA's
//    softmax and its start and end overlap the others' copies.  (Three stages and
//    two CTAs took 8 % more, one V stage and four CTAs 41 %.)
//  * V rows past the context are zeroed in shared memory (0 * NaN).  Waits are
//    bounded (2 s); after a timeout the softmax warps keep walking the tiles
//    without waiting, so that their barriers stay matched.
#pragma once

#include <stddef.h>

#include "pa_decode_kernel.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kTcTile = 128;               // tokens per tile
constexpr uint32_t kTcStage = 16384;       // 128 tokens x 128 codes
constexpr float kTcSlack = 3.f;            // log2 units a score may exceed the reference by
constexpr float kTcPShift = 12.f;          // log2 of what P is scaled by: [0, 8] -> [0, 2^15], e5m2's top binade

// Heads' rows of one term, for GT query heads: of Q (two terms), and of P (three).
constexpr int tc_q_heads(int gt) { return gt <= 8 ? 8 : 16; }
constexpr int tc_p_heads(int gt) { return gt <= 4 ? 4 : gt <= 8 ? 8 : 16; }
// P's columns (a multiple of 16), and the bytes of one of its two buffers: whole 8-row
// atoms of the rows that there are.  (The MMAs read 8 rows past the last of 24: of the
// next buffer, or of Q behind it; their columns of O are never read.)
constexpr int tc_p_cols(int gt) { return (3 * tc_p_heads(gt) + 15) / 16 * 16; }
constexpr uint32_t tc_p_bytes(int gt) { return (3u * tc_p_heads(gt) + 7u) / 8u * 1024u; }

template <int NH, int HP>
struct TcShared {
  uint64_t full_k[2], full_v[2], empty_k[2], empty_v[2], s[2], p[2], pv[2], scl_full[2], drain;
  // scales (K's, log2 of V's) of the 128 / bs <= 16 blocks of tile j, HP heads each, in
  // slot j & 1: tile j+2's are written when its V stage is free, which is after P_j
  alignas(16) float scl[2][2][16 * HP];
  alignas(16) float mx[4][NH];             // per warp: tile maximum of every head; at the end, sums
  alignas(16) float wx[4][NH];             // likewise of z
  uint32_t tmem_base;
  int abort;
};

template <int GT, int HP>
constexpr uint32_t tc_smem_bytes() {
  return 4 * kTcStage + 2 * tc_p_bytes(GT) + 2u * tc_q_heads(GT) * 128u +
         (uint32_t)sizeof(TcShared<tc_q_heads(GT), HP>) + 1024u;
}
// (three CTAs of up to 8 heads per SM: 228 KB less 1 KB a CTA that the system takes)
static_assert(tc_smem_bytes<8, 1>() <= 75 * 1024 && tc_smem_bytes<8, 4>() <= 75 * 1024, "three CTAs per SM");

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
// kind::f8f6f4, A e4m3 (format 0), B e4m3 or e5m2 (format 1), fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn_major, bool b_e5m2) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Two floats as e4m3 codes (a in the low byte), saturating, and back.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void from_e4m3x2(uint32_t c, float& a, float& b) {
  uint32_t h;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(c));
  f16x2_to_float2(h, a, b);
}
// The same for e5m2 codes, which are the upper bytes of f16 values.
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void from_e5m2x2(uint32_t c, float& a, float& b) {
  f16x2_to_float2(__byte_perm(c, 0u, 0x1404), a, b);
}
__device__ __forceinline__ void sts_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Barrier 2 of the 128 softmax threads, true for all if true for any.
__device__ __forceinline__ bool vote128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(x ? 1u : 0u) : "memory");
  return r != 0;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(smem_u32(bar), parity)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity)) return true;
  atomicOr(&g_status_decode, PA_DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}
// Byte x of row n of a 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t swz_byte(int n, int x) {
  return (uint32_t)(n * 128 + (((x >> 4) ^ (n & 7)) << 4) + (x & 15));
}

// The score (log2 units) of query head hq for sequence b's token t, by itself.
template <int D>
__device__ __noinline__ float plain_score(const DecodeParams& p, int b, int t, int hq, int kvh) {
  int id = p.block_tables[(size_t)b * p.max_blocks + t / p.bs];
  if ((unsigned)id >= (unsigned)p.num_blocks) id = 0;
  const uint8_t* k = p.k_codes + (((size_t)id * p.bs + t % p.bs) * p.Hkv + kvh) * D;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)b * p.Hq + hq) * D;
  float acc = 0.f, m = 0.f;
  for (int d = 0; d < D; ++d) m = fmaxf(m, fabsf(__bfloat162float(q[d])));
  const int e = query_exponent(m);
  for (int d = 0; d < D; ++d) {
    __nv_fp8_e4m3 c;
    c.__x = k[d];
    acc = fmaf(__bfloat162float(q[d]) * pow2i(-e), static_cast<float>(c), acc);
  }
  return acc * (p.qscale * pow2i(e) * p.k_scale[(size_t)id * p.scale_row + kvh]);
}

// GT: query heads of the CTA, rounded up (1, 2, 4, 8, 16); HP: KV heads per row
// of 128 codes; W: weights mode.  p.nsub CTAs share the HP * G query heads of a
// row's KV heads, hs = ceil(HP * G / nsub) each.
template <int GT, int HP, bool W>
__global__ void __launch_bounds__(kTcThreads, GT <= 8 ? 3 : 2)
tc_decode_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const DecodeParams p) {
  constexpr int D = 128 / HP;
  constexpr int NH = tc_q_heads(GT), N = 2 * NH;     // Q's rows and the columns of S
  constexpr int NP = tc_p_heads(GT), NO = tc_p_cols(GT);
  constexpr uint32_t kTmem = GT <= 8 ? 64u : 128u;   // S_0, S_1: N columns each, O: NO
  static_assert(2 * N + NO <= (int)kTmem, "tensor memory");
  constexpr uint32_t kPBytes = tc_p_bytes(GT);
  constexpr uint32_t kOffV = 2 * kTcStage, kOffP = 4 * kTcStage, kOffQ = kOffP + 2 * kPBytes;
  static_assert(NO * 128u - kPBytes <= N * 128u, "P's MMAs read inside the tiles");
  using Shared = TcShared<NH, HP>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Shared* sh = reinterpret_cast<Shared*>(smem + kOffQ + N * 128);
  volatile int* abort_flag = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- item: KV heads innermost (neighbouring CTAs read neighbouring rows of the same blocks),
  // partitions outermost (the CTAs without work, past the shorter contexts, come last)
  int u = (int)blockIdx.x;
  const int rowh = u % (p.Hkv / HP);            // row of 128 codes: KV heads rowh * HP and on
  u /= p.Hkv / HP;
  const int sub = u % p.nsub;
  u /= p.nsub;
  const int b = u % p.B, part = u / p.B;
  const int Lmax = p.max_blocks * p.bs;
  const int hs = (HP * p.G + p.nsub - 1) / p.nsub;
  const int h0 = rowh * HP * p.G + sub * hs;    // first query head
  const int gh = min(hs, HP * p.G - sub * hs);  // query heads of this CTA, <= GT (0: the last one is short)
  // which of the row's KV heads query head h reads
  auto kv_of = [&](int h) -> int { return HP == 1 ? 0 : (sub * hs + min(h, gh - 1)) / p.G; };
  const int t0 = part * p.part_tokens;
  const int bsh = 31 - __clz(p.bs);
  // What does not depend on the context's length is requested with it: the
  // queries, and the first five tiles' block-table entries (a lane each, inside
  // the row whatever the length is).
  __nv_bfloat16 qraw[GT];
  int id[5] = {0, 0, 0, 0, 0};
  if (warp < 4) {
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)b * p.Hq + h0) * D;
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      const int d = (int)threadIdx.x - kv_of(h) * D;       // the thread's column within the head, if it has one
      qraw[h] = gh > 0 && (HP == 1 || (d >= 0 && d < D)) ? qp[min(h, gh - 1) * D + d] : __float2bfloat16_rn(0.f);
    }
  } else if (warp == 4) {
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int i = ((t0 + j * kTcTile) >> bsh) + lane;
      if (lane < (kTcTile >> bsh) && i < p.max_blocks) id[j] = __ldg(&p.block_tables[(size_t)b * p.max_blocks + i]);
    }
  }
  const int L0 = __ldg(&p.context_lens[b]);
  const int L = L0 < 0 ? 0 : min(L0, Lmax);
  if (part == 0 && rowh == 0 && sub == 0 && threadIdx.x == 0 && L != L0) atomicOr(&g_status_decode, PA_DEV_BAD_LEN);
  const int nparts = L > 0 ? (L + p.part_tokens - 1) / p.part_tokens : 1;
  if (part >= nparts || gh <= 0) return;        // nothing allocated yet
  const int t1 = min(L, t0 + p.part_tokens);
  const int nt = (t1 - t0 + kTcTile - 1) / kTcTile;

  // ---- TMA producer, its state and first requests: the ring is empty, so the first two tiles
  // go out before the CTA has met at its barrier
  const uint64_t pol = policy_evict_first();
  const uint32_t box = (uint32_t)p.bs * 128u;
  auto in_use = [&](int j) -> bool {
    return j < nt && lane < (kTcTile >> bsh) && t0 + j * kTcTile + (lane << bsh) < t1;
  };
  auto boxes_of = [&](int j) -> int { return (min(kTcTile, t1 - t0 - j * kTcTile) + p.bs - 1) >> bsh; };
  auto checked = [&](int id) -> int {
    if ((unsigned)id < (unsigned)p.num_blocks) return id;
    atomicOr(&g_status_decode, PA_DEV_BAD_BLOCK);
    return 0;                                   // keep every copy inside the pool
  };
  auto request = [&](const CUtensorMap& map, uint64_t* full, uint32_t off, int j, int blk) {
    const int nb = boxes_of(j);
    if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)nb * box);
    __syncwarp();
    if (lane < nb) tma_load_4d(smem + off + (j & 1) * kTcStage + lane * box, &map, full, 0, rowh, 0, blk, pol);
  };
  const int first = min(nt, 2);
  if (warp == 4) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh->full_k[i], 1);
        mbar_init(&sh->full_v[i], 1);
        mbar_init(&sh->empty_k[i], 1);
        mbar_init(&sh->empty_v[i], 1);
        mbar_init(&sh->s[i], 1);
        mbar_init(&sh->p[i], 128);
        mbar_init(&sh->pv[i], 1);
      }
      for (int i = 0; i < 2; ++i) mbar_init(&sh->scl_full[i], 1);
      mbar_init(&sh->drain, 1);
      sh->abort = 0;
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j) id[j] = in_use(j) ? checked(id[j]) : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (j < first) request(mapK, &sh->full_k[j], 0, j, id[j]);
    if (first > 0) request(mapV, &sh->full_v[0], kOffV, 0, id[0]);
  }
  __syncwarp();
  float qf[GT];                                  // scale * log2(e) * 2^e of every head
  if (warp < 4) {
    // ---- Q: two e4m3 rows per head, while the first tiles are on their way
    float q[GT];
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      q[h] = __bfloat162float(qraw[h]);
      const float m = warp_max(fabsf(q[h]));
      if (lane == 0) sh->mx[warp][h] = m;
    }
    named_sync(1, 128);
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      const float m = fmaxf(fmaxf(sh->mx[0][h], sh->mx[1][h]), fmaxf(sh->mx[2][h], sh->mx[3][h]));
      const int e = query_exponent(m);
      // (an infinite query has no answer: NaN, as its scores would be)
      const float x = m < INFINITY ? q[h] * pow2i(-e) : NAN;
      qf[h] = p.qscale * pow2i(e);
      const uint32_t hi = e4m3x2(x, 0.f);
      float back, none;
      from_e4m3x2(hi, back, none);
      const uint32_t lo = e4m3x2((x - back) * 16.f, 0.f);
      sts_u8(sbase + kOffQ + swz_byte(h, (int)threadIdx.x), hi);
      sts_u8(sbase + kOffQ + swz_byte(NH + h, (int)threadIdx.x), lo);
    }
    fence_proxy_async_smem();
  }
  if (warp == 5) {
    tmem_alloc(&sh->tmem_base, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const uint32_t tO = tmem + 2 * N;

  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    const int32_t* row = p.block_tables + (size_t)b * p.max_blocks;
    // Lane i: block i of a tile (at most 16), its id and scales.  The scales hang
    // on the id and both come from memory: ids are read three tiles ahead and
    // scales two, so that neither latency is waited for (one tile ahead for
    // both held every tile up by two memory latencies, about 4000 clocks).
    struct Scales {
      float k[HP], v[HP];
    };
    auto scales_of = [&](int id) -> Scales {
      Scales x;
#pragma unroll
      for (int i = 0; i < HP; ++i) {
        x.k[i] = __ldg(&p.k_scale[(size_t)id * p.scale_row + rowh * HP + i]);
        x.v[i] = __ldg(&p.v_scale[(size_t)id * p.scale_row + rowh * HP + i]);   // (its log2 when it is used)
      }
      return x;
    };
    auto put_scales = [&](int j, const Scales& x) {
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < HP; ++i) {
          sh->scl[j & 1][0][lane * HP + i] = x.k[i];
          sh->scl[j & 1][1][lane * HP + i] = log2f(x.v[i]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->scl_full[j & 1]);
    };
    if (first > 1) request(mapV, &sh->full_v[1], kOffV, 1, id[1]);
    const Scales sc_0 = scales_of(id[0]), sc_1 = scales_of(id[1]);
    int blk = in_use(2) ? checked(id[2]) : 0;
    Scales sc = scales_of(blk);
    int blk1 = in_use(3) ? checked(id[3]) : 0;
    Scales sc1 = scales_of(blk1);
    int blk2 = id[4];
    if (first > 0) put_scales(0, sc_0);
    if (first > 1) put_scales(1, sc_1);
    int issued_k = first, issued_v = first;
    for (int j = 2; j < nt; ++j) {
      const int st = j & 1;
      const uint32_t ph = ((uint32_t)(j >> 1) & 1u) ^ 1u;
      if (!__all_sync(0xffffffffu, tc_wait(&sh->empty_k[st], ph, abort_flag))) break;
      request(mapK, &sh->full_k[st], 0, j, blk);
      issued_k = j + 1;
      if (!__all_sync(0xffffffffu, tc_wait(&sh->empty_v[st], ph, abort_flag))) break;
      request(mapV, &sh->full_v[st], kOffV, j, blk);
      issued_v = j + 1;
      put_scales(j, sc);
      blk = blk1;
      sc = sc1;
      blk1 = in_use(j + 2) ? checked(blk2) : 0;
      sc1 = scales_of(blk1);
      blk2 = in_use(j + 3) ? __ldg(&row[((t0 + (j + 3) * kTcTile) >> bsh) + lane]) : 0;
    }
    // no TMA write may land after the CTA has left
    if (lane == 0) {
      for (int j = max(0, issued_k - 2); j < issued_k; ++j) mbar_wait(&sh->full_k[j & 1], (uint32_t)(j >> 1) & 1u);
      for (int j = max(0, issued_v - 2); j < issued_v; ++j) mbar_wait(&sh->full_v[j & 1], (uint32_t)(j >> 1) & 1u);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idS = idesc_e4m3_f32(kTcTile, N, false, false);
      constexpr uint32_t idO = idesc_e4m3_f32(128, NO, true, true);
      const uint64_t dk = sdesc_sw128(sbase, 16, 1024), dq = sdesc_sw128(sbase + kOffQ, 16, 1024);
      const uint64_t dv = sdesc_sw128(sbase + kOffV, kTcStage, 1024), dp = sdesc_sw128(sbase + kOffP, 16, 1024);
      auto issue_s = [&](int j) {
        const uint64_t dkj = sdesc_at(dk, (uint32_t)(j & 1) * kTcStage);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)           // 32 head dims each
          umma_f8(tmem + (j & 1) * N, sdesc_at(dkj, kk * 32u), sdesc_at(dq, kk * 32u), idS, kk > 0 ? 1u : 0u);
        umma_commit(&sh->s[j & 1]);
        umma_commit(&sh->empty_k[j & 1]);
      };
      if (tc_wait(&sh->full_k[0], 0, abort_flag)) {
        tc_fence_after();
        issue_s(0);
        for (int j = 0; j < nt; ++j) {
          const int st = j & 1;
          const uint32_t ph = (uint32_t)(j >> 1) & 1u;
          if (j + 1 < nt) {
            if (!tc_wait(&sh->full_k[(j + 1) & 1], (uint32_t)((j + 1) >> 1) & 1u, abort_flag)) break;
            tc_fence_after();
            issue_s(j + 1);
          }
          if (!tc_wait(&sh->p[st], ph, abort_flag)) break;
          if (!tc_wait(&sh->full_v[st], ph, abort_flag)) break;
          tc_fence_after();
          const uint64_t dvj = sdesc_at(dv, (uint32_t)st * kTcStage), dpj = sdesc_at(dp, (uint32_t)st * kPBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)         // 32 tokens each: four 8-token groups of 1024 bytes
            umma_f8(tO, sdesc_at(dvj, kk * 4096u), sdesc_at(dpj, kk * 32u), idO, (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&sh->pv[st]);
          umma_commit(&sh->empty_v[st]);
        }
      }
      umma_commit(&sh->drain);                   // every MMA has completed before TMEM is freed
      mbar_wait(&sh->drain, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int r = (int)threadIdx.x;              // token of the tile, head dim at either end; TMEM lane
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    float m[GT], l[GT], w[GT];
    int kvi[GT];
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      m[h] = w[h] = -INFINITY;
      l[h] = 0.f;
      kvi[h] = kv_of(h);
    }
    // x[kv] for a head's kv without indexing registers
    auto pick = [&](const float (&x)[HP], int kv) -> float {
      float y = x[0];
#pragma unroll
      for (int i = 1; i < HP; ++i) y = kv == i ? x[i] : y;
      return y;
    };

    for (int j = 0; j < nt; ++j) {
      const int st = j & 1;
      const uint32_t ph = (uint32_t)(j >> 1) & 1u;
      const int t = t0 + j * kTcTile + r;
      const bool ok = t < t1;
      tc_wait(&sh->scl_full[st], ph, abort_flag);
      float ks[HP], lv[HP];
#pragma unroll
      for (int i = 0; i < HP; ++i) {
        ks[i] = sh->scl[st][0][(r >> bsh) * HP + i];
        lv[i] = ok ? sh->scl[st][1][(r >> bsh) * HP + i] : -INFINITY;
      }
      __syncwarp();
      tc_wait(&sh->s[st], ph, abort_flag);
      __syncwarp();
      tc_fence_after();
      float s[GT];
      {
        uint32_t hi[NH], lo[NH];
        if constexpr (NH == 8) {
          uint32_t v[16];
          tmem_ld16(tmem + st * N + lane_off, v);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            hi[h] = v[h];
            lo[h] = v[8 + h];
          }
        } else {
          uint32_t v[32];
          tmem_ld32(tmem + st * N + lane_off, v);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            hi[h] = v[h];
            lo[h] = v[16 + h];
          }
        }
#pragma unroll
        for (int h = 0; h < GT; ++h)
          s[h] = ok ? fmaf(__uint_as_float(lo[h]), 0.0625f, __uint_as_float(hi[h])) * (qf[h] * pick(ks, kvi[h])) : -INFINITY;
      }
      if constexpr (HP > 1) {
        // a NaN code of another KV head in the row times this head's zeros is NaN:
        // such a token's scores are taken from its own codes
#pragma unroll
        for (int h = 0; h < GT; ++h)
          if (s[h] != s[h]) s[h] = plain_score<D>(p, b, t, h0 + min(h, gh - 1), rowh * HP + kvi[h]);
      }
      if constexpr (W) {
        if (ok) {
          float* sp = p.ws_s + ((size_t)b * p.Hq + h0) * (size_t)Lmax + t;
#pragma unroll
          for (int h = 0; h < GT; ++h)
            if (h < gh) sp[(size_t)h * Lmax] = s[h];
        }
      }
      // z is kept where a head's scale has to be picked from several (64 x 8 heads in groups of 4 over
      // U[1024, 8192]: head_dim 64 79 -> 77 us, 32 117 -> 104); with one scale an addition is
      // cheaper than the register (groups of 8 over head_dim 128: 121 against 123)
      bool need = false;
      float z[GT];
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        if constexpr (HP > 1) {
          z[h] = s[h] + pick(lv, kvi[h]);
          need = need || s[h] > m[h] + kTcSlack || z[h] > w[h] + kTcSlack;
        } else {
          need = need || s[h] > m[h] + kTcSlack || s[h] + lv[0] > w[h] + kTcSlack;
        }
      }
      __syncwarp();
      if (vote128(need)) {
        // new references: the tile's maxima where they are above
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float x = warp_max(s[h]), y = warp_max(HP > 1 ? z[h] : s[h] + lv[0]);
          if (lane == 0) {
            sh->mx[warp][h] = x;
            sh->wx[warp][h] = y;
          }
        }
        named_sync(1, 128);
        float f[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float x = fmaxf(fmaxf(sh->mx[0][h], sh->mx[1][h]), fmaxf(sh->mx[2][h], sh->mx[3][h]));
          const float y = fmaxf(fmaxf(sh->wx[0][h], sh->wx[1][h]), fmaxf(sh->wx[2][h], sh->wx[3][h]));
          const float mn = fmaxf(m[h], x), wn = fmaxf(w[h], y);
          l[h] *= m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn);
          f[h] = w[h] == -INFINITY ? 0.f : exp2f(w[h] - wn);
          m[h] = mn;
          w[h] = wn;
        }
        if (j > 0) {
          // O holds V_{j-1} P_{j-1}: this thread's head dim, every head's three columns
          tc_wait(&sh->pv[(j - 1) & 1], (uint32_t)((j - 1) >> 1) & 1u, abort_flag);
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            uint32_t v[NP];
            tmem_ld(tO + i * NP + lane_off, v);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < GT; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * f[h]);
            tmem_st(tO + i * NP + lane_off, v);
          }
          tmem_st_wait();
        }
        named_sync(1, 128);                      // mx is free again
      }
      // P: 2^(z - w + 12) as three e5m2 terms, byte r of rows h, NP + h and 2 NP + h
      const uint32_t pb = sbase + kOffP + (uint32_t)st * kPBytes;
      auto weight = [&](int h) -> float {
        const float x = HP > 1 ? z[h] : s[h] + lv[0];
        return x == -INFINITY ? 0.f : exp2f(x - w[h] + kTcPShift);
      };
#pragma unroll
      for (int h = 0; h < GT; h += 2) {
        l[h] += s[h] == -INFINITY ? 0.f : exp2f(s[h] - m[h]);
        if constexpr (GT > 1) l[h + 1] += s[h + 1] == -INFINITY ? 0.f : exp2f(s[h + 1] - m[h + 1]);
        const float x0 = weight(h), x1 = GT > 1 ? weight(h + (GT > 1)) : 0.f;
        float r0 = x0, r1 = x1;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint32_t c = e5m2x2(r0, r1);
          sts_u8(pb + swz_byte(i * NP + h, r), c);
          if constexpr (GT > 1) sts_u8(pb + swz_byte(i * NP + h + 1, r), c >> 8);
          float y0, y1;
          from_e5m2x2(c, y0, y1);
          // 16 (r - y), exactly
          f2unpack(ffma2(f2pack(y0, y1), f2pack(-16.f, -16.f), fmul2(f2pack(r0, r1), f2pack(16.f, 16.f))), r0, r1);
        }
      }
      if (!ok) {
        // the slot may hold anything (NaN codes, an older tile): 0 * NaN would reach O
        tc_wait(&sh->full_v[st], ph, abort_flag);
        unsigned char* vrow = smem + kOffV + st * kTcStage + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vrow + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&sh->p[st]);
    }

    // ------------------------------------------------------------ output
    __syncwarp();
    named_sync(1, 128);
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      float x = l[h];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (lane == 0) sh->mx[warp][h] = x;
    }
    named_sync(1, 128);
    float o[GT];
#pragma unroll
    for (int h = 0; h < GT; ++h) o[h] = 0.f;
    if (nt > 0) {
      tc_wait(&sh->pv[(nt - 1) & 1], (uint32_t)((nt - 1) >> 1) & 1u, abort_flag);
      __syncwarp();
      tc_fence_after();
      auto up = [&](int h) -> float { return w[h] == -INFINITY ? 0.f : exp2f(w[h] - m[h] - kTcPShift); };
      uint32_t v[3][NP];
#pragma unroll
      for (int i = 0; i < 3; ++i) tmem_ld(tO + i * NP + lane_off, v[i]);
      tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < GT; ++h)
        o[h] = fmaf(fmaf(__uint_as_float(v[2][h]), 0.0625f, __uint_as_float(v[1][h])), 0.0625f, __uint_as_float(v[0][h])) *
               up(h);
    }
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      if (h >= gh) break;
      const float den = (sh->mx[0][h] + sh->mx[1][h]) + (sh->mx[2][h] + sh->mx[3][h]);
      const size_t bh = (size_t)b * p.Hq + h0 + h;
      const size_t slot = bh * p.max_parts + part;
      const int d = r - kvi[h] * D;              // the row's columns of the head's own KV head
      if (HP == 1 || (d >= 0 && d < D)) {
        if (nparts > 1)
          p.ws_o[slot * D + d] = o[h];
        else
          static_cast<__nv_bfloat16*>(p.out)[bh * D + d] = __float2bfloat16_rn(den != 0.f ? o[h] / den : 0.f);
      }
      if (r == 0 && (W || nparts > 1)) {
        p.ws_ml[slot * 2] = m[h];
        p.ws_ml[slot * 2 + 1] = den;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kTmem);
}

}  // namespace
}  // namespace pa
