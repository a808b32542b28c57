// pa_prefill_fp8_blocks.cu — causal attention of each sequence's newest tokens
// over an e4m3 pool with one scale per (block, KV head).
//
// Row i of sequence b (n_b rows, the last n_b tokens of its context) sits at
// position p = L_b - n_b + i and attends to the keys at 0..p:
//   out = sum_t softmax_t(scale * <q, K_t>) V_t,  K = value(code) * k_scale[block, head], V likewise.
//
// tile_kernel (head_dim 128, blocks of 8 and more): 5th-generation tensor cores.  One CTA per (pair of
// query tiles, KV head), one CTA per SM: a tile is 128 rows = QP = 128 / G positions
// x G query heads; keys in tiles of 128; scores and output in tensor memory.
//  * S = Q K^T takes the codes of K as they are (kind::f8f6f4).  Q enters as two terms,
//    hi in e4m3 and lo in e5m2: q 2^-e = hi + lo with 2^e per row so that the row's
//    largest value is in [128, 256).  hi takes 4 significant bits of a bf16 value and
//    leaves 4, at most 8 units of the value's last place, which e5m2's 3 bits hold
//    exactly: the split is exact down to 2^-13 of the largest, and within 2^-20 of it below.
//    (lo in e4m3 ends at 2^-9, so it dropped what is below 2^-17 of the largest.)  K's
//    scales stay apart, in the softmax.
//  * P V runs in bf16: a weight is off by at most 2^-8 of itself, either way, so that the
//    output's error against 64 bits is 0.0023 of it where the last rounding alone makes
//    0.0017.  (bf16 has fp32's range: no weight is lost.  8-bit terms of P, as in
//    decode, would be three products of the larger kind.)  V's codes come by TMA into a stage of their own; warps 8-11
//    widen them (codes_to_bf16), multiply their scale in (one rounding to bf16, none for a
//    power of two; bf16 has the exponents for it, so a row that attends only to blocks of
//    small scale keeps its precision beside blocks of large scale) and write the 128-byte-swizzled
//    tile that both query tiles' MMAs read: widening a tile is as many instructions as
//    its softmax, and the pair shares it.
//  * One thread per row (warps 0-3 and 4-7, a query tile each): x = s * (K scale of
//    the key's block) * (row factor), running maximum and sum, P = 2^(x - m) in bf16
//    over the S columns.  The reference only moves when the maximum has grown by 2^8.
//  * A query tile goes in steps of 64 keys.  Tensor memory is full: two buffers of 64
//    columns for S (then P) and an O of 128 for each query tile.  Warps 13 and 14 issue
//    a query tile's MMAs each: P V of a step, then the S of the next but one, so that
//    the step's successor has its scores already.  (Steps of 128 keys in one buffer
//    make less of the tensor core wait for its A operand, 68 clocks an MMA against 48
//    for half the work, but chain softmax, P V and S: 14 % slower on 8 chunks of 512
//    queries.  One issuing warp for both tiles: 8 % more on top, its waits in a row.)
//  * What bounds it: a step of a query tile is a chain of softmax, P V, S and the waits
//    between them, and the MMAs' operands take most of the shared memory's bandwidth.
//    8 chunks of 512 queries x 32 heads (8 KV heads) over U[1024, 4096] take 170 us
//    (910 TFLOP/s, 48 % of the library's bf16 rate); a mixed round of 16 sequences with
//    1 to 100 new tokens each 43 to 45.  The softmax spills 136 bytes at 128 registers.
//  * Keys at or past the context length have P = 0, and in the V tile they are finite
//    whatever the pool holds: a NaN code comes out finite, a block past the context with
//    a scale of 0.  A NaN of a key in the context has to reach the rows at and past it
//    and no others of its tile: the first such key of each head dim is noted and makes
//    NaN of that dim at the end.  Every wait is bounded (2 s).
//
// rows_kernel: one warp per (row, query head), for the other sizes.  Lane t of a step of
// 32 keys computes one key's whole score from its row of codes; the warp takes
// the running maximum and sum, then every lane accumulates its D / 32 head
// dims over the 32 keys.  The block's K scale multiplies the score, its V scale
// the softmax weight; the sum of the softmax is over the unscaled weights.
#include <float.h>
#include <limits.h>
#include <stddef.h>

#include "pa_tc.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_prefill_fp8;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRowWarps = 4;

struct Params {
  void* out;
  const void* q;
  const int32_t* query_start;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int B, rows, Hq, Hkv, G, D, bs, max_blocks, num_blocks, scale_row;
  float qscale;                 // scale * log2(e)
};

// Whether sequence b's rows lie in [0, rows] in order.
__device__ __forceinline__ bool good_rows(const Params& p, int b) {
  const int a = __ldg(&p.query_start[b]), e = __ldg(&p.query_start[b + 1]);
  return a >= 0 && e >= a && e <= p.rows;
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const Params p) {
  __shared__ float qs[kRowWarps][D];
  constexpr int DPL = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x;
  const int hq = (int)blockIdx.y * kRowWarps + warp;
  if (row == 0 && blockIdx.y == 0) {
    for (int i = (int)threadIdx.x; i < p.B; i += kRowWarps * 32) {
      const int L = __ldg(&p.context_lens[i]);
      if (!good_rows(p, i) || L < 0 || L > p.max_blocks * p.bs) atomicOr(&g_status_prefill_fp8, PA_DEV_BAD_LEN);
    }
  }
  if (hq >= p.Hq) return;
  const int b = find_unit(p.query_start, p.B, 1, 0, row);   // the last sequence that starts at or before the row
  if (!good_rows(p, b)) return;
  const int r0 = __ldg(&p.query_start[b]), r1 = __ldg(&p.query_start[b + 1]);
  if (row < r0 || row >= r1) return;
  int L = __ldg(&p.context_lens[b]);
  L = L < 0 ? 0 : min(L, p.max_blocks * p.bs);
  const int pos = L - (r1 - r0) + (row - r0);
  const int h = hq / p.G;
  const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)row * p.Hq + hq) * D;
  float qmax = 0.f;
  for (int d = lane; d < D; d += 32) qmax = fmaxf(qmax, fabsf(__bfloat162float(qrow[d])));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, off));
  const int qe = query_exponent(qmax);
  const float rowf = p.qscale * pow2i(qe);
  for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(qrow[d]) * pow2i(-qe);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) o[d] = 0.f;
  const size_t tok = (size_t)p.Hkv * D;
  const int32_t* tab = p.block_tables + (size_t)b * p.max_blocks;
  for (int k0 = 0; k0 <= pos; k0 += 32) {
    const int t = k0 + lane;
    float s = -INFINITY, vs = 0.f;
    size_t at = 0;
    if (t <= pos) {
      int blk = __ldg(&tab[t / p.bs]);
      if ((unsigned)blk >= (unsigned)p.num_blocks) {
        atomicOr(&g_status_prefill_fp8, PA_DEV_BAD_BLOCK);
        blk = 0;
      }
      at = ((size_t)blk * p.bs + t % p.bs) * tok + (size_t)h * D;
      float acc = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float f[16];
        Elem<fp8e4m3>::unpack(__ldg(reinterpret_cast<const uint4*>(p.k + at) + c), f);
#pragma unroll
        for (int e = 0; e < 16; ++e) acc = fmaf(qs[warp][16 * c + e], f[e], acc);
      }
      s = acc * (rowf * __ldg(&p.k_scale[(size_t)blk * p.scale_row + h]));
      vs = __ldg(&p.v_scale[(size_t)blk * p.scale_row + h]);
    }
    float mx = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    mx = fmaxf(mx, m);
    const float alpha = mx == -INFINITY ? 1.f : exp2f(m - mx);
    m = mx;
    l *= alpha;
#pragma unroll
    for (int d = 0; d < DPL; ++d) o[d] *= alpha;
    const float pk = s == -INFINITY ? 0.f : exp2f(s - m);
    l += pk;
    const float pw = pk * vs;
    const int cnt = min(32, pos - k0 + 1);
    for (int i = 0; i < cnt; ++i) {
      const float w = __shfl_sync(0xffffffffu, pw, i);
      const size_t vat = __shfl_sync(0xffffffffu, (unsigned long long)at, i);
      const uint8_t* vp = p.v + vat + lane * DPL;
#pragma unroll
      for (int d = 0; d < DPL; ++d) {
        __nv_fp8_e4m3 c;
        c.__x = __ldg(vp + d);
        o[d] = fmaf(w, static_cast<float>(c), o[d]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  const float inv = l != 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + ((size_t)row * p.Hq + hq) * D + lane * DPL;
#pragma unroll
  for (int d = 0; d < DPL; ++d) orow[d] = __float2bfloat16_rn(o[d] * inv);
}


// ------------------------------------------------------------------ tile_kernel

constexpr int kTileThreads = 480;      // 2 x 4 softmax, 4 V, TMA and 2 MMA warps
constexpr int kRows = 128;
constexpr int kKT = 128;               // keys per tile
constexpr int kStep = 64;              // keys per step of a query tile
constexpr int kKStages = 3;
constexpr uint32_t kQHalf = 16384;     // 128 rows x 128 bytes
constexpr uint32_t kCodes = 16384;     // 128 keys x 128 codes
constexpr uint32_t kVHalf = 16384;     // 128 keys x 64 columns of bf16
constexpr uint32_t kOffQ = 0;          // 2 query tiles x (bf16 columns 0-63, 64-127; then hi, lo; at the end the output)
constexpr uint32_t kOffK = 65536;      // 3 stages of codes
constexpr uint32_t kOffV = 114688;     // 2 stages x 2 halves of bf16
constexpr uint32_t kOffRawV = 180224;  // 2 stages of codes
constexpr uint32_t kOffBar = 212992;
constexpr uint32_t kTileSmem = kOffBar + 3072 + 1024;   // + alignment slack
constexpr int kSorted = 128;           // batches up to which the longest contexts' pairs come first
constexpr float kRescaleThreshold = 8.0f;               // log2 units
constexpr uint32_t kTmemCols = 512;    // query tile h: S (and P) at columns 128 h, O at 256 + 128 h

struct Bars {
  uint64_t q[2], qf[2], full_k[kKStages], empty_k[kKStages], raw_v[2], raw_ev[2], full_v[2], empty_v[2];
  uint64_t s[2][2], p[2][2], pv[2], scl_full[4], drain[2];
  // K scale of every 4 keys (block sizes are multiples of 4) of tile t in slot
  // t & 3: those of t+1 to t+3 may be written while the softmax reads t's, t+4's
  // only after P_t (its K stage waits for S_{t+1}, which is issued after P_t)
  alignas(16) float kscl[4][kKT / 4];
  float kup[4];                          // what tile t's scales are to be multiplied by: 1, or 2^32
  // first key whose V is NaN, of every head dim, and whether there is any
  int nan_key[128];
  int any_nan;
  // the batch's context lengths and pairs, and the sequence and pair of this CTA
  int len[kSorted], pairs[kSorted], seq, pair;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 3072 && offsetof(Bars, kscl) % 16 == 0, "barrier block");

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(smem_u32(bar), parity)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity)) return true;
  atomicOr(&g_status_prefill_fp8, PA_DEV_TIMEOUT);
  *abort_flag = 1;
  return false;
}
__device__ __forceinline__ float ex2_f32(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// D[tmem] (+)= A[smem] * B[smem], 8-bit operands of the descriptor's formats.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
// Four floats as e4m3 codes (the first in the low byte).
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// The same as e5m2 codes.
__device__ __forceinline__ uint32_t to_e5m2x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e5m2x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ void from_e4m3x4(uint32_t c, float* f) {
  uint32_t a, b;
  e4m3x4_to_f16x2x2(c, a, b);
  f16x2_to_float2(a, f[0], f[1]);
  f16x2_to_float2(b, f[2], f[3]);
}

// Four codes' bits 7: set for a NaN (the other bits say nothing).
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
// The NaN among the sixteen codes of key t, head dims d and on.
__device__ __noinline__ void note_nan(uint4 c, Bars* bars, int d, int t, int kend) {
  if (t >= kend) return;
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    for (uint32_t m = nan_bits(w[k]) & 0x80808080u; m; m &= m - 1) {
      atomicMin(&bars->nan_key[d + 4 * k + ((__ffs(m) - 1) >> 3)], t);
      bars->any_nan = 1;
    }
  }
}
// Four codes times s (bf16 in both halves) as bf16 pairs.  A code's seven magnitude bits, taken for
// the last four of a bf16's exponent and the first three of its digits, are its value times 2^-120,
// the subnormal ones too; two products put that right and the scale in (one factor s 2^120 would
// overflow for s >= 2^8).  A NaN code comes out as 480 s: finite, so that 0 times it is 0.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t s, uint32_t& a, uint32_t& b) {
  const uint32_t hi = ((w >> 4) & 0x07070707u) | (w & 0x80808080u), lo = (w << 4) & 0xf0f0f0f0u;
  constexpr uint32_t kUp = 0x7b807b80u;                  // 2^120
  a = mul_bf16x2(mul_bf16x2(__byte_perm(lo, hi, 0x5140), kUp), s);
  b = mul_bf16x2(mul_bf16x2(__byte_perm(lo, hi, 0x7362), kUp), s);
}

// Sixteen codes times a scale that bf16 does not hold: the products in fp32, rounded once.
struct Row16 {
  uint4 a, b;
};
__device__ __noinline__ Row16 scaled_row(uint4 c, float s) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    codes_to_bf16(w[k], 0x3f803f80u, o[2 * k], o[2 * k + 1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(bf16lo(o[2 * k + e]) * s, bf16hi(o[2 * k + e]) * s);
      o[2 * k + e] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  return {make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7])};
}

// V (four warps): the codes of each key tile as bf16 rows.  Thread x takes the
// 16-code chunk x % 8 of rows x / 8, x / 8 + 16, ...
__device__ __forceinline__ void convert_v(const Params& p, Bars* bars, unsigned char* smem, int b, int kvh, int kend,
                                          int nt, int x) {
  constexpr int RS = 16;
  volatile int* abort_flag = &bars->abort;
  const int lane = (int)(threadIdx.x & 31);
  const int ch = x & 7, r0 = x >> 3;
  const float* scales = p.v_scale + kvh;
  const int32_t* tab = p.block_tables + (size_t)b * p.max_blocks;
  const int bsh = 31 - __clz(p.bs), nbt = kKT >> bsh;    // blocks per tile, a lane each: at most 32
  // codes 16 ch .. 16 ch + 15 are columns of half ch / 4, 16-byte chunks 2 (ch % 4) and the next
  unsigned char* tile = smem + kOffV + (ch >> 2) * kVHalf;
  const int c0 = (ch & 3) * 2;
  auto id_of = [&](int t) -> int {                       // -1: no block of the context
    if (t < nt && lane < nbt && t * kKT + (lane << bsh) < kend) {
      const int id = __ldg(&tab[((t * kKT) >> bsh) + lane]);
      return (unsigned)id < (unsigned)p.num_blocks ? id : 0;   // (flagged by the TMA warp)
    }
    return -1;
  };
  // its bits; 0 past the context, where codes may be anything and P is 0
  auto scale_of = [&](int id) -> uint32_t {
    return __float_as_uint(id >= 0 ? __ldg(&scales[(size_t)id * p.scale_row]) : 0.f);
  };
  // scales (a lane each) of the tile at hand and of the next, block ids of the one after
  int id2 = -1;
  uint32_t sc0 = 0u, sc1 = 0u;
  if (nt > 0) {
    const int id0 = id_of(0), id1 = id_of(1);
    id2 = id_of(2);
    sc0 = scale_of(id0);
    sc1 = scale_of(id1);
  }
  for (int t = 0; t < nt; ++t) {
    const int st = t & 1;
    const uint32_t ph = (uint32_t)(t >> 1) & 1u;
    bool ok = wait_or_abort(&bars->empty_v[st], ph ^ 1u, abort_flag);
    ok = ok && wait_or_abort(&bars->raw_v[st], ph, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) break;
    const unsigned char* from = smem + kOffRawV + st * kCodes + ch * 16;
    unsigned char* dst = tile + st * 2 * kVHalf;
    // a scale is a bf16 as it stands (every power of two is) when its lower half is empty
    const bool bf16_scales = !__any_sync(0xffffffffu, (sc0 & 0xffffu) != 0u);
    // four rows at a time, read before the first is written (the compiler keeps
    // shared-memory reads behind writes: one by one a row took a latency each)
#pragma unroll 1
    for (int rr = r0; rr < kKT; rr += 4 * RS) {
      uint4 c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = *reinterpret_cast<const uint4*>(from + (rr + i * RS) * 128);
      // bit 7 of a byte's magnitude plus one: set for the NaN code (0x7f, 0xff) alone
      uint32_t bad = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        bad |= nan_bits(c[i].x) | nan_bits(c[i].y) | nan_bits(c[i].z) | nan_bits(c[i].w);
      if (bad & 0x80808080u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) note_nan(c[i], bars, ch * 16, t * kKT + rr + i * RS, kend);
      }
      if (!bf16_scales) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = rr + i * RS;
          const Row16 o = scaled_row(c[i], __uint_as_float(__shfl_sync(0xffffffffu, sc0, r >> bsh)));
          *reinterpret_cast<uint4*>(dst + r * 128 + ((c0 ^ (r & 7)) << 4)) = o.a;
          *reinterpret_cast<uint4*>(dst + r * 128 + (((c0 + 1) ^ (r & 7)) << 4)) = o.b;
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = rr + i * RS;
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t o[8];
        const uint32_t s2 = __byte_perm(__shfl_sync(0xffffffffu, sc0, r >> bsh), 0u, 0x3232);
#pragma unroll
        for (int k = 0; k < 4; ++k) codes_to_bf16(w[k], s2, o[2 * k], o[2 * k + 1]);
        *reinterpret_cast<uint4*>(dst + r * 128 + ((c0 ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + r * 128 + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&bars->full_v[st]);
    mbar_arrive(&bars->raw_ev[st]);
    sc0 = sc1;
    sc1 = scale_of(id2);
    id2 = id_of(t + 3);
  }
}

__global__ void __launch_bounds__(kTileThreads, 1)
tile_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapO,
            const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV, const Params p,
            const int QP) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item.  Up to kSorted sequences: the longest context first, so that what the SMs end
  // with is short (8 chunks of 512: 193 us in the batch's order, 180 in this; a mixed round 54, 47).
  // More, of which the SMs take many turns: sequence b's pairs are units U_b = floor(query_start[b] / (2 QP)) + b
  // and on; n rows make at most floor(n / (2 QP)) + 1 pairs, which never passes U_{b+1}
  const int kvh = (int)(blockIdx.x % p.Hkv);
  const int u = (int)(blockIdx.x / p.Hkv);
  if (blockIdx.x == 0) {
    for (int i = (int)threadIdx.x; i < p.B; i += kTileThreads) {
      const int Li = __ldg(&p.context_lens[i]);
      if (!good_rows(p, i) || Li < 0 || Li > p.max_blocks * p.bs) atomicOr(&g_status_prefill_fp8, PA_DEV_BAD_LEN);
    }
  }
  int b, pi;
  if (p.B <= kSorted) {
    const int x = (int)threadIdx.x;
    int mine = 0, len = 0;
    if (x < p.B) {
      len = __ldg(&p.context_lens[x]);
      mine = good_rows(p, x) ? (__ldg(&p.query_start[x + 1]) - __ldg(&p.query_start[x]) + 2 * QP - 1) / (2 * QP) : 0;
      bars->len[x] = len;
      bars->pairs[x] = mine;
    }
    if (x == 0) bars->seq = -1;
    __syncthreads();
    if (x < p.B) {
      int before = 0;                              // pairs of the longer contexts
      for (int i = 0; i < p.B; ++i)
        if (bars->len[i] > len || (bars->len[i] == len && i < x)) before += bars->pairs[i];
      if (u >= before && u < before + mine) {
        bars->seq = x;
        bars->pair = u - before;
      }
    }
    __syncthreads();
    b = bars->seq;
    if (b < 0) return;
    pi = bars->pair;
  } else {
    b = find_unit(p.query_start, p.B, 2 * QP, 1, u);
    if (!good_rows(p, b)) return;
    pi = u - (__ldg(&p.query_start[b]) / (2 * QP) + b);
  }
  const int qrow0 = __ldg(&p.query_start[b]);
  const int nq = __ldg(&p.query_start[b + 1]) - qrow0;
  const int npairs = (nq + 2 * QP - 1) / (2 * QP);
  if (pi < 0 || pi >= npairs) return;              // nothing allocated yet
  int L = __ldg(&p.context_lens[b]);
  L = L < 0 ? 0 : min(L, p.max_blocks * p.bs);
  // query tile h: rows q0 + h QP and on; its keys [0, kend_h), none if it has no rows
  const int q0 = (npairs - 1 - pi) * 2 * QP;       // the longest pair first
  auto kend_of = [&](int h) -> int {
    const int first = q0 + h * QP;
    return first < nq ? max(0, min(L, L - nq + min(first + QP, nq))) : 0;
  };
  const int kend = max(kend_of(0), kend_of(1));
  // key tiles of the pair, and steps of 64 keys of each query tile
  const int nt = (kend + kKT - 1) / kKT;
  const int ns0 = (kend_of(0) + kStep - 1) / kStep, ns1 = (kend_of(1) + kStep - 1) / kStep;

  if (threadIdx.x == 384) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bars->q[h], 1);
      mbar_init(&bars->qf[h], 128);
      mbar_init(&bars->raw_v[h], 1);
      mbar_init(&bars->raw_ev[h], 128);
      mbar_init(&bars->full_v[h], 128);
      mbar_init(&bars->empty_v[h], 2);
      mbar_init(&bars->drain[h], 1);
      mbar_init(&bars->s[h][0], 1);
      mbar_init(&bars->s[h][1], 1);
      mbar_init(&bars->p[h][0], 128);
      mbar_init(&bars->p[h][1], 128);
      mbar_init(&bars->pv[h], 1);
    }
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bars->full_k[i], 1);
      mbar_init(&bars->empty_k[i], 2);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars->scl_full[i], 1);
    bars->abort = 0;
    bars->any_nan = 0;
    fence_mbar_init();
    prefetch_tensormap(&mapQ);
    const uint64_t pol = policy_evict_first();
    for (int h = 0; h < 2; ++h) {
      if ((h ? ns1 : ns0) == 0) continue;
      unsigned char* dst = smem + kOffQ + h * 2 * kQHalf;
      mbar_arrive_expect_tx(&bars->q[h], 2u * 128u * (uint32_t)(p.G * QP));
      tma_load_4d(dst, &mapQ, &bars->q[h], 0, kvh * p.G, qrow0 + q0 + h * QP, 0, pol);
      tma_load_4d(dst + kQHalf, &mapQ, &bars->q[h], 64, kvh * p.G, qrow0 + q0 + h * QP, 0, pol);
    }
  }
  __syncwarp();
  if (threadIdx.x < 128) bars->nan_key[threadIdx.x] = INT_MAX;
  if (warp == 13) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp >= 8 && warp < 12) {
    convert_v(p, bars, smem, b, kvh, kend, nt, (int)threadIdx.x - 256);
  } else if (warp == 12) {
    // ---------------------------------------------------------- code requests, K's scales
    const int32_t* tab = p.block_tables + (size_t)b * p.max_blocks;
    const int bsh = 31 - __clz(p.bs), nbt = kKT >> bsh;    // blocks per tile, a lane each
    const uint32_t box = (uint32_t)p.bs * 128u;
    const uint64_t pol = policy_evict_last();              // other query tiles read the same codes
    if (lane == 0) {
      prefetch_tensormap(&mapK);
      prefetch_tensormap(&mapV);
    }
    auto id_of = [&](int t) -> int {
      const bool used = t < nt && lane < nbt && t * kKT + (lane << bsh) < kend;
      return used ? __ldg(&tab[((t * kKT) >> bsh) + lane]) : 0;
    };
    auto checked = [&](int id) -> int {
      if ((unsigned)id < (unsigned)p.num_blocks) return id;
      atomicOr(&g_status_prefill_fp8, PA_DEV_BAD_BLOCK);
      return 0;
    };
    auto scale_of = [&](int id) -> float { return __ldg(&p.k_scale[(size_t)id * p.scale_row + kvh]); };
    int issued_k = 0, issued_v = 0;
    int id = checked(id_of(0)), id1 = checked(id_of(1)), id2 = id_of(2);
    float sc = scale_of(id), sc1 = scale_of(id1);
    int ks = 0;                                            // K stage, and its use count's parity
    uint32_t kph = 1u;
    for (int t = 0; t < nt; ++t) {
      const int nb = (min(kKT, kend - t * kKT) + p.bs - 1) >> bsh;
      bool ok = true;
      if (lane == 0) ok = wait_or_abort(&bars->empty_k[ks], kph, abort_flag);
      if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars->full_k[ks], (uint32_t)nb * box);
      __syncwarp();
      if (lane < nb) tma_load_4d(smem + kOffK + ks * kCodes + lane * box, &mapK, &bars->full_k[ks], 0, kvh, 0, id, pol);
      issued_k = t + 1;
      // a scale of 0 as the tiniest one: the scores are 0 all the same, and a masked -inf stays one;
      // a tile with scales so large that their products with raw scores (up to 2^24) could be past
      // fp32's range, where small queries bring them back, holds them times 2^-32
      const bool big = __any_sync(0xffffffffu, sc > 0x1p96f);
      const float ks4 = __shfl_sync(0xffffffffu, sc, (4 * lane) >> bsh) * (big ? 0x1p-32f : 1.f);
      bars->kscl[t & 3][lane] = fmaxf(ks4, __uint_as_float(1u));
      if (lane == 0) bars->kup[t & 3] = big ? 0x1p32f : 1.f;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars->scl_full[t & 3]);
        ok = wait_or_abort(&bars->raw_ev[t & 1], ((uint32_t)(t >> 1) & 1u) ^ 1u, abort_flag);
      }
      if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars->raw_v[t & 1], (uint32_t)nb * box);
      __syncwarp();
      if (lane < nb)
        tma_load_4d(smem + kOffRawV + (t & 1) * kCodes + lane * box, &mapV, &bars->raw_v[t & 1], 0, kvh, 0, id, pol);
      issued_v = t + 1;
      id = id1;
      sc = sc1;
      id1 = checked(id2);
      sc1 = scale_of(id1);
      id2 = id_of(t + 3);
      if (++ks == kKStages) {
        ks = 0;
        kph ^= 1u;
      }
    }
    // no TMA write may land after the CTA has left
    if (lane == 0) {
      for (int t = max(0, issued_k - kKStages); t < issued_k; ++t)
        mbar_wait(&bars->full_k[t % kKStages], (uint32_t)(t / kKStages) & 1u);
      for (int t = max(0, issued_v - 2); t < issued_v; ++t) mbar_wait(&bars->raw_v[t & 1], (uint32_t)(t >> 1) & 1u);
      if (ns0 > 0) mbar_wait(&bars->q[0], 0);
      if (ns1 > 0) mbar_wait(&bars->q[1], 0);
    }
  } else if (warp >= 13) {
    // ---------------------------------------------------------- MMA issuers, one per query tile
    if (lane == 0 && nt > 0) {
      // fp32 scores of e4m3 keys; of Q the e4m3 term, then the e5m2 one (format 1 of A)
      constexpr uint32_t idHi = (1u << 4) | ((uint32_t)(kStep >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
      constexpr uint32_t idLo = idHi | (1u << 7);
      constexpr uint32_t idO = idesc_bf16_f32(kRows, 128, false, true);   // V MN-major
      const int h = warp - 13, ns = h ? ns1 : ns0;
      const uint64_t dq = sdesc_sw128(sbase + kOffQ + h * 2 * kQHalf, 16, 1024), dk = sdesc_sw128(sbase + kOffK, 16, 1024);
      const uint64_t dv = sdesc_sw128(sbase + kOffV, kVHalf, 1024);
      const uint32_t tS = tmem + h * 128, tO = tmem + 256 + h * 128;
      int ks = 0;                                          // stage of the next scores' key tile, and its parity
      uint32_t kph = 0u;
      // scores of step i: hi, then lo, 32 head dims each.  A query tile that has no more
      // steps keeps giving back the stages.
      auto scores = [&](int i) -> bool {
        const int g = i & 1;
        if (g == 0 && !wait_or_abort(&bars->full_k[ks], kph, abort_flag)) return false;
        if (i < ns) {
          tc_fence_after();
          const uint64_t dkj = sdesc_at(dk, (uint32_t)ks * kCodes + (uint32_t)g * (kStep * 128u));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_f8(tS + g * 64, sdesc_at(dq, (uint32_t)(kk >> 2) * kQHalf + (uint32_t)(kk & 3) * 32u),
                    sdesc_at(dkj, (uint32_t)(kk & 3) * 32u), kk < 4 ? idHi : idLo, kk > 0 ? 1u : 0u);
          umma_commit(&bars->s[h][g]);
        }
        if (g == 1) {
          umma_commit(&bars->empty_k[ks]);
          if (++ks == kKStages) {
            ks = 0;
            kph ^= 1u;
          }
        }
        return true;
      };
      bool ok = (ns == 0 || wait_or_abort(&bars->qf[h], 0, abort_flag)) && scores(0) && scores(1);
      for (int i = 0; i < 2 * nt && ok; ++i) {
        const int t = i >> 1, g = i & 1;
        if (g == 0) ok = wait_or_abort(&bars->full_v[t & 1], (uint32_t)(t >> 1) & 1u, abort_flag);
        if (i < ns) {
          ok = ok && wait_or_abort(&bars->p[h][g], (uint32_t)t & 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dvj = sdesc_at(dv, (uint32_t)(t & 1) * 2 * kVHalf + (uint32_t)g * 8192u);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_ts(tO, tS + g * 64 + kk * 8, sdesc_at(dvj, (uint32_t)kk * 2048u), idO, (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars->pv[h]);
        }
        if (!ok) break;
        if (g == 1) umma_commit(&bars->empty_v[t & 1]);
        if (i + 2 < 2 * nt) ok = scores(i + 2);
      }
      // every MMA issued so far has completed before TMEM is freed
      umma_commit(&bars->drain[h]);
      mbar_wait(&bars->drain[h], 0);
    }
  } else {
    // ---------------------------------------------------------- softmax + epilogue
    const int h = warp >> 2;                       // query tile of the pair
    const int r = (warp & 3) * 32 + lane;          // tile row and TMEM lane
    const int qi = r / p.G, hh = r % p.G;
    const int qt = q0 + h * QP;                    // the tile's first row in the sequence
    const int pos = L - nq + qt + qi;
    const int ns = h ? ns1 : ns0;
    const bool row_out = qi < QP && (qt + qi) < nq;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + h * 128 + lane_off, tO = tmem + 256 + h * 128 + lane_off;
    unsigned char* qs = smem + kOffQ + h * 2 * kQHalf + r * 128;   // the row's two halves
    float rowf = 0.f;                              // scale * log2(e) * the row's power of two
    bool live = true;
    if (ns > 0) {
      // this thread's row of Q, in place: bf16 halves -> hi and lo; zeros for rows that are not the sequence's
      live = __all_sync(0xffffffffu, wait_or_abort(&bars->q[h], 0, abort_flag));
      uint4 qv[16];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        qv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live && row_out)
          qv[i] = *reinterpret_cast<const uint4*>(qs + (i >> 3) * kQHalf + (((i & 7) ^ (r & 7)) << 4));
        float f[8];
        Elem<__nv_bfloat16>::unpack(qv[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
      }
      const int qe = query_exponent(mx);
      // (an infinite query has no answer: NaN, as its scores would be)
      const float down = mx < INFINITY ? pow2i(-qe) : NAN;
      rowf = fmaxf(p.qscale * pow2i(qe), FLT_MIN);
#pragma unroll
      for (int i = 0; i < 8; ++i) {                // 16 head dims
        float f[16];
        Elem<__nv_bfloat16>::unpack(qv[2 * i], f);
        Elem<__nv_bfloat16>::unpack(qv[2 * i + 1], f + 8);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float* x = f + 4 * e;
          float y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] *= down;
          hi[e] = to_e4m3x4(x[0], x[1], x[2], x[3]);
          from_e4m3x4(hi[e], y);
          lo[e] = to_e5m2x4(x[0] - y[0], x[1] - y[1], x[2] - y[2], x[3] - y[3]);
        }
        if (live) {
          *reinterpret_cast<uint4*>(qs + ((i ^ (r & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(qs + kQHalf + ((i ^ (r & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      if (live) mbar_arrive(&bars->qf[h]);
    }
    float m_ref = -INFINITY, lsum = 0.f;
    for (int j = 0; j < ns && live; ++j) {
      const int g = j & 1, t = j >> 1;             // step j: half g of key tile t
      const int k0 = j * kStep;
      const uint32_t tP = tS + g * 64;
      bool ok = g == 1 || wait_or_abort(&bars->scl_full[t & 3], (uint32_t)(t >> 2) & 1u, abort_flag);
      ok = ok && wait_or_abort(&bars->s[h][g], (uint32_t)t & 1u, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
      tc_fence_after();
      const float4* ks4 = reinterpret_cast<const float4*>(bars->kscl[t & 3]) + 4 * g;   // 16 keys' scales each
      const bool partial = k0 + kStep - 1 > pos;
      // maximum of the row's scaled scores, 32 keys at a time
      const float rf = rowf * bars->kup[t & 3];
      float mx = -INFINITY;
      uint32_t buf[2][32];
      tmem_ld32(tP, buf[0]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t (&v)[32] = buf[c];
        tmem_ld_wait();
        if (c < 1) tmem_ld32(tP + 32, buf[1]);
        if (partial) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (k0 + c * 32 + i > pos) v[i] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 k4 = ks4[2 * c + i];
          const float f[4] = {k4.x, k4.y, k4.z, k4.w};
          float a[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t* x = &v[i * 16 + 4 * g];
            a[g] = f[g] * fmax3(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), __uint_as_float(x[2]),
                                __uint_as_float(x[3]));
          }
          mx = fmax3(fmax3(mx, a[0], a[1]), a[2], a[3]);
        }
      }
      mx *= rf;
      const bool need = mx > m_ref + kRescaleThreshold;
      const float alpha = need ? exp2f(m_ref - mx) : 1.f;
      if (need) m_ref = mx;
      if (j > 0 && __any_sync(0xffffffffu, need)) {
        ok = wait_or_abort(&bars->pv[h], (uint32_t)(j - 1) & 1u, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t w[16];
          tmem_ld16(tO + c * 16, w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
          tmem_st16(tO + c * 16, w);
        }
        tmem_st_wait();
      }
      lsum *= alpha;
      const float negm = m_ref == -INFINITY ? 0.f : -m_ref;
      const uint64_t nm2 = f2pack(negm, negm);
      uint64_t ls2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ls2[i] = f2pack(0.f, 0.f);
      // P of keys 32 c .. 32 c + 31 into columns 16 c .. 16 c + 15
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t (&v)[32] = buf[c];
        uint32_t pw[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 k4 = ks4[2 * c + (i >> 3)];
          const int q = (i >> 1) & 3;
          // (above 0: a masked score is -inf, and -inf * 0 is NaN)
          const float f = fmaxf(rf * (q == 0 ? k4.x : q == 1 ? k4.y : q == 2 ? k4.z : k4.w), FLT_MIN);
          float x0, x1;
          f2unpack(ffma2(f2pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2pack(f, f), nm2), x0, x1);
          const float p0 = ex2_f32(x0), p1 = ex2_f32(x1);
          const __nv_bfloat162 pk = __floats2bfloat162_rn(p0, p1);
          ls2[i & 3] = fadd2(ls2[i & 3], f2pack(p0, p1));
          pw[i] = *reinterpret_cast<const uint32_t*>(&pk);
        }
        tmem_st16(tP + c * 16, pw);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->p[h][g]);
      float ls8[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) f2unpack(ls2[i], ls8[2 * i], ls8[2 * i + 1]);
      lsum += ((ls8[0] + ls8[1]) + (ls8[2] + ls8[3])) + ((ls8[4] + ls8[5]) + (ls8[6] + ls8[7]));
    }

    bool have = ns > 0 && live;
    if (have) {
      // (the last scores were there before the last but one P V: that phase has to pass first)
      bool ok = ns < 2 || wait_or_abort(&bars->pv[h], (uint32_t)(ns - 2) & 1u, abort_flag);
      ok = ok && wait_or_abort(&bars->pv[h], (uint32_t)(ns - 1) & 1u, abort_flag);
      have = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    const float inv = lsum != 0.f ? 1.f / lsum : 0.f;
    const bool full = ns > 0 && qt + QP <= nq;
    const bool nan_values = have && *static_cast<volatile int*>(&bars->any_nan);
    unsigned char* orow = static_cast<unsigned char*>(p.out) +
                          (((size_t)qrow0 + qt + qi) * p.Hq + (size_t)kvh * p.G + hh) * 256;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t v[32];
      if (have) {
        tmem_ld32(tO + c * 32, v);
        tmem_ld_wait();
      }
      if (nan_values) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (*static_cast<volatile int*>(&bars->nan_key[c * 32 + i]) <= pos) v[i] = 0x7fffffffu;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = have ? __uint_as_float(v[g * 8 + 2 * e]) * inv : 0.f;
          const float a1 = have ? __uint_as_float(v[g * 8 + 2 * e + 1]) * inv : 0.f;
          const __nv_bfloat162 pk = __floats2bfloat162_rn(a0, a1);
          w[e] = *reinterpret_cast<const uint32_t*>(&pk);
        }
        const int ch = c * 4 + g;
        if (full) {
          // staged in the tile's Q buffer (free: its last S completed before its last P V) for two TMA stores
          *reinterpret_cast<uint4*>(qs + (ch >> 3) * kQHalf + (((ch & 7) ^ (r & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        } else if (row_out) {
          st_v4(orow + ch * 16, make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
    }
    if (full) {
      fence_proxy_async_smem();
      named_sync(1 + h, 128);
      if ((warp & 3) == 0 && lane == 0) {
        unsigned char* src = smem + kOffQ + h * 2 * kQHalf;
        tma_store_4d(&mapO, src, 0, kvh * p.G, qrow0 + qt, 0);
        tma_store_4d(&mapO, src + kQHalf, 64, kvh * p.G, qrow0 + qt, 0);
        bulk_commit();
        bulk_wait_all();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

unsigned* status_word_prefill_fp8_blocks() { return device_word(g_status_prefill_fp8); }

}  // namespace pa

using namespace pa;

extern "C" int pa_prefill_fp8_blocks(void* out, const void* query, const int32_t* query_start, int total_queries,
                                     const void* k_cache, const void* v_cache, const float* k_scale,
                                     const float* v_scale, const int32_t* block_tables, int max_blocks_per_seq,
                                     const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                                     int head_dim, int block_size, int num_blocks, float scale, pa_dtype dtype,
                                     void* stream) {
  if (dtype != PA_BF16) return PA_ERR_DTYPE;
  if (num_seqs < 0 || total_queries < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads ||
      num_blocks <= 0 || max_blocks_per_seq <= 0 || !supported_head_dim(head_dim) ||
      !supported_block_size(block_size) || !(scale > 0.f) ||
      (long long)max_blocks_per_seq * block_size > kMaxRowTokens)
    return PA_ERR_SHAPE;
  const long long groups = ((long long)num_heads + kRowWarps - 1) / kRowWarps;
  if (groups > 65535) return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_queries == 0) return PA_OK;
  if (!out || !query || !query_start || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens)
    return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
      !aligned16(v_scale))
    return PA_ERR_ALIGN;
  Params p;
  p.out = out;
  p.q = query;
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.B = num_seqs;
  p.rows = total_queries;
  p.Hq = num_heads;
  p.Hkv = num_kv_heads;
  p.G = num_heads / num_kv_heads;
  p.D = head_dim;
  p.bs = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.scale_row = scale_row(num_kv_heads);
  p.qscale = scale * kLog2e;
  if (head_dim == 128 && block_size >= 8 && p.G <= kRows) {   // (K's boxes are whole 8-row swizzle atoms)
    const int QP = kRows / p.G;
    const long long ctas = ((long long)total_queries / (2 * QP) + num_seqs) * num_kv_heads;
    if (ctas > 0x7fffffffll) return PA_ERR_SHAPE;
    CUtensorMap mapQ, mapO, mapK, mapV;
    const uint64_t dims[4] = {128, (uint64_t)num_heads, (uint64_t)total_queries, 1};
    const uint64_t str[3] = {256, (uint64_t)num_heads * 256, (uint64_t)total_queries * num_heads * 256};
    const uint32_t box[4] = {64, (uint32_t)p.G, (uint32_t)QP, 1};
    if (!encode_map(&mapQ, query, PA_BF16, 4, dims, str, box, true) ||
        !encode_map(&mapO, out, PA_BF16, 4, dims, str, box, true)) {
      note_host_error("cuTensorMapEncodeTiled failed for the query tile");
      return PA_ERR_CUDA;
    }
    int dev = 0;
    if (!ck(cudaGetDevice(&dev), "cudaGetDevice")) return PA_ERR_CUDA;
    // K's codes 128-byte-swizzled for the MMAs, V's plain
    if (!pool_map(&mapK, k_cache, PA_FP8_E4M3, num_blocks, block_size, num_kv_heads, 128, dev, true, 1) ||
        !pool_map(&mapV, v_cache, PA_FP8_E4M3, num_blocks, block_size, num_kv_heads, 128, dev, false, 1)) {
      note_host_error("cuTensorMapEncodeTiled failed for the K/V pool");
      return PA_ERR_CUDA;
    }
    if (!raise_smem_limit(reinterpret_cast<const void*>(&tile_kernel), dev)) return PA_ERR_CUDA;
    int qp = QP;
    void* args[] = {&mapQ, &mapO, &mapK, &mapV, &p, &qp};
    if (!ck(cudaLaunchKernel(reinterpret_cast<const void*>(&tile_kernel), dim3((unsigned)ctas), dim3(kTileThreads),
                             args, kTileSmem, (cudaStream_t)stream),
            "cudaLaunchKernel(tile_kernel)"))
      return PA_ERR_CUDA;
    return PA_OK;
  }
  const dim3 grid((unsigned)total_queries, (unsigned)groups);
  if (head_dim == 128)
    rows_kernel<128><<<grid, kRowWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else if (head_dim == 64)
    rows_kernel<64><<<grid, kRowWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else
    rows_kernel<32><<<grid, kRowWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return ck(cudaGetLastError(), "launch rows_kernel") ? PA_OK : PA_ERR_CUDA;
}
