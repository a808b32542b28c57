// pa_decode_direct.cuh — paged decode attention on CUDA cores with the cache read
// straight into registers, for any head_dim, block_size and query group; pools of
// f32, bf16 or e4m3 codes with one scale per (block, KV head).  Shared by the
// translation units that instantiate it.
//
// One CTA = (sequence, partition, KV head, up to GT query heads).  LPT lanes share
// a token, each with 4 (f32) or 8 elements of head_dim; a warp takes kU = 4 passes of
// 32 / LPT tokens at a time: their block ids were read a step ahead, the K and V
// rows of all of them are requested together (8 loads of 8 or 16 bytes in flight
// per lane), then come the scores, one update of the running maximum for the lot,
// and the weighted sum over V.  Nothing is staged and nothing is waited for but
// the loads, so a short context costs its chain of memory latencies (lengths, ids,
// rows) and no pipeline's fill: with few and short requests that chain is the call.
// Lane groups and warps are merged by log-sum-exp at the end.
// Arithmetic is fp32 throughout.
// 5 requests x 4 KV heads of head_dim 64 (f32, groups of 3) of up to 700 tokens take
// 10 us on the GPU with their weights, 41 through the TMA ring of decode_kernel, whose
// fill such contexts never repay; 32 x 8 heads of 128 over U[128, 4096]: bf16 in
// groups of 7 163 us against 140, so at large batches the ring is 15 % ahead.
// What bounds large calls: over e4m3, instruction issue (35 requests x 21 heads of 64 in
// groups of 3, 106 us: 0.67 a cycle and scheduler, widening and shuffles beside the
// products); over f32 in large groups the latency of loads (18 requests x 4 heads of 128
// in groups of 16, 622 to 632 us: issue 0.38, waiting for memory the top stall, DRAM 7 %
// busy: the four CTAs of a group each read K and V, three of them from L2).
#pragma once

#include "pa_decode_kernel.cuh"

namespace pa {
namespace {

constexpr int kDirectWarps = kDirectThreads / 32;

// Elements per lane, and a lane's load of them.
template <typename KT> struct DirectLoad;
template <> struct DirectLoad<float> {
  static constexpr int kE = 4;
  using Raw = uint4;
  __device__ __forceinline__ static Raw load(const unsigned char* p) { return ld_nc_v4(p); }
  __device__ __forceinline__ static void unpack(const Raw& r, float* f) { Elem<float>::unpack(r, f); }
};
template <> struct DirectLoad<__nv_bfloat16> {
  static constexpr int kE = 8;
  using Raw = uint4;
  __device__ __forceinline__ static Raw load(const unsigned char* p) { return ld_nc_v4(p); }
  __device__ __forceinline__ static void unpack(const Raw& r, float* f) { Elem<__nv_bfloat16>::unpack(r, f); }
};
template <> struct DirectLoad<fp8e4m3b> {
  static constexpr int kE = 8;
  using Raw = uint2;
  __device__ __forceinline__ static Raw load(const unsigned char* p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
  }
  __device__ __forceinline__ static void unpack(const Raw& r, float* f) {
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t a, b;
      e4m3x4_to_f16x2x2(w[i], a, b);
      f16x2_to_float2(a, f[4 * i], f[4 * i + 1]);
      f16x2_to_float2(b, f[4 * i + 2], f[4 * i + 3]);
    }
  }
};

// T: query/output type; KT: pool type; GT: query heads of the CTA, rounded up
// (p.nsub CTAs share a group's G, ceil(G / nsub) each); W: weights mode.
// One head over codes of up to 64 dims: held to 64 registers, eight CTAs per SM (64 x 5
// heads of 64 over U[1024, 8192]: 62 us, 70 at the compiler's own 72).
template <typename T, typename KT, int D, int GT, bool W>
__global__ void __launch_bounds__(kDirectWarps * 32, (sizeof(KT) == 1 && GT == 1 && D <= 64) ? 8 : 0)
direct_decode_kernel(const DecodeParams p, const unsigned char* __restrict__ k_cache,
                     const unsigned char* __restrict__ v_cache) {
  using E = Elem<T>;
  using DL = DirectLoad<KT>;
  constexpr int EB = Elem<KT>::kBytes, KE = DL::kE;
  constexpr int LPT = D / KE, TPW = 32 / LPT;
  // four query heads of 8 elements a lane leave registers for half the passes (at
  // four: 168 registers, three CTAs per SM)
  constexpr int kU = GT == 4 && KE == 8 ? 2 : 4;
  // packed pairs once several heads share the widened elements (e4m3 blocks of 4,
  // group 4: 195 -> 152 us; one head over bf16: 217 -> 235 us, the packing alone)
  constexpr bool kPairs = GT > 1;
  constexpr int STEP = kDirectWarps * kU * TPW;         // tokens of a CTA step
  constexpr bool BLK = std::is_same<KT, fp8e4m3b>::value;
  static_assert(LPT >= 4 && LPT <= 32, "lane split");
  __shared__ float so[kDirectWarps][GT][D], sm[kDirectWarps][GT], sl[kDirectWarps][GT], up[kDirectWarps][GT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane / LPT, li = lane % LPT;
  asm volatile("griddepcontrol.launch_dependents;");

  // subgroups innermost (they read the same rows), partitions outermost
  int u = (int)blockIdx.x;
  const int sub = u % p.nsub;
  u /= p.nsub;
  const int kvh = u % p.Hkv;
  u /= p.Hkv;
  const int b = u % p.B, part = u / p.B;
  const int Lmax = p.max_blocks * p.bs;
  const int hs = (p.G + p.nsub - 1) / p.nsub;
  const int h0 = kvh * p.G + sub * hs, gh = min(hs, p.G - sub * hs);
  if (gh <= 0) return;
  const int t0 = part * p.part_tokens;
  const int bsh = 31 - __clz(p.bs);
  const int32_t* tab = p.block_tables + (size_t)b * p.max_blocks;
  // pass k of step i: token t0 + i * STEP + (k * kDirectWarps + warp) * TPW + grp
  auto token = [&](int i, int k) -> int { return t0 + i * STEP + (k * kDirectWarps + warp) * TPW + grp; };
  // requested with the length: the queries, and the first step's block ids (inside the row in any case)
  int id[kU];
#pragma unroll
  for (int k = 0; k < kU; ++k) id[k] = __ldg(&tab[min(token(0, k), Lmax - 1) >> bsh]);
  float q[GT][KE];
#pragma unroll
  for (int h = 0; h < GT; ++h) {
    const T* qp = static_cast<const T*>(p.q) + ((size_t)b * p.Hq + h0 + min(h, gh - 1)) * D + li * KE;
#pragma unroll
    for (int j = 0; j < KE / E::kPerChunk; ++j)
      E::unpack(__ldg(reinterpret_cast<const uint4*>(qp) + j), &q[h][j * E::kPerChunk]);
  }
  const int L0 = __ldg(&p.context_lens[b]);
  const int L = L0 < 0 ? 0 : min(L0, Lmax);
  if (L != L0 && part == 0 && kvh == 0 && sub == 0 && threadIdx.x == 0) atomicOr(&g_status_decode, PA_DEV_BAD_LEN);
  const int nparts = L > 0 ? (L + p.part_tokens - 1) / p.part_tokens : 1;
  if (part >= nparts) return;
  const int t1 = min(L, t0 + p.part_tokens);
  const int ns = (t1 - t0 + STEP - 1) / STEP;
  // Over codes, a query past 2^64 or below 2^-64 has its size go with the block's scale: its sums of
  // products with codes may be past fp32's range where the scale brings them back.  (Every query:
  // 3 % more, a product a token and head.)
  bool far = false;
  if constexpr (BLK) {
    float mx[GT];
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      mx[h] = 0.f;
#pragma unroll
      for (int e = 0; e < KE; ++e) mx[h] = fmaxf(mx[h], fabsf(q[h][e]));
#pragma unroll
      for (int off = LPT / 2; off > 0; off >>= 1) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], off));
      far = far || mx[h] > 0x1p64f || (mx[h] > 0.f && mx[h] < 0x1p-64f);
    }
    if (far) {
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        const int x = query_exponent(mx[h]);
#pragma unroll
        for (int e = 0; e < KE; ++e) q[h][e] *= pow2i(-x);
        if (lane == 0) up[warp][h] = pow2i(x);
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < GT; ++h)
#pragma unroll
    for (int e = 0; e < KE; ++e) q[h][e] *= p.qscale;

  float m[GT], l[GT], o[GT][KE];
#pragma unroll
  for (int h = 0; h < GT; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < KE; ++e) o[h][e] = 0.f;
  }
  const size_t tok = (size_t)p.Hkv * D * EB;
  const size_t col = (size_t)kvh * D * EB + (size_t)li * KE * EB;
  for (int i = 0; i < ns; ++i) {
    typename DL::Raw kr[kU], vr[kU];
    float ks[kU], vs[kU];
    bool ok[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int t = token(i, k);
      ok[k] = t < t1;
      int blk = id[k];
      if (ok[k] && (unsigned)blk >= (unsigned)p.num_blocks) {
        atomicOr(&g_status_decode, PA_DEV_BAD_BLOCK);
        blk = 0;
      }
      if (!ok[k]) blk = 0;                 // (block 0 is read and not used: no load hangs on a branch)
      const size_t at = (((size_t)blk << bsh) + (t & (p.bs - 1))) * tok + col;
      kr[k] = DL::load(k_cache + at);
      vr[k] = DL::load(v_cache + at);
      ks[k] = BLK ? __ldg(&p.k_scale[(size_t)blk * p.scale_row + kvh]) : 1.f;
      vs[k] = BLK ? __ldg(&p.v_scale[(size_t)blk * p.scale_row + kvh]) : 1.f;
    }
    if (i + 1 < ns) {
#pragma unroll
      for (int k = 0; k < kU; ++k) id[k] = __ldg(&tab[min(token(i + 1, k), Lmax - 1) >> bsh]);
    }
    float s[kU][GT];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      float f[KE];
      DL::unpack(kr[k], f);
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        float a = 0.f;
        if constexpr (kPairs) {
          uint64_t a2 = f2pack(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < KE; e += 2) a2 = ffma2(f2pack(q[h][e], q[h][e + 1]), f2pack(f[e], f[e + 1]), a2);
          float a1;
          f2unpack(a2, a, a1);
          a += a1;
        } else {
#pragma unroll
          for (int e = 0; e < KE; ++e) a = fmaf(q[h][e], f[e], a);
        }
#pragma unroll
        for (int off = LPT / 2; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
        s[k][h] = a;
      }
    }
    if (BLK && far) {
#pragma unroll
      for (int k = 0; k < kU; ++k)
#pragma unroll
        for (int h = 0; h < GT; ++h) s[k][h] *= ks[k] * up[warp][h];
    } else if constexpr (BLK) {
#pragma unroll
      for (int k = 0; k < kU; ++k)
#pragma unroll
        for (int h = 0; h < GT; ++h) s[k][h] *= ks[k];
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        s[k][h] = ok[k] ? s[k][h] : -INFINITY;
        if constexpr (W) {
          if (li == 0 && ok[k] && h < gh)
            p.ws_s[((size_t)b * p.Hq + h0 + h) * (size_t)Lmax + token(i, k)] = s[k][h];
        }
      }
    }
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      float mx = m[h];
#pragma unroll
      for (int k = 0; k < kU; ++k) mx = fmaxf(mx, s[k][h]);
      const float a = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mx);
      m[h] = mx;
      l[h] *= a;
#pragma unroll
      for (int e = 0; e < KE; ++e) o[h][e] *= a;
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (!ok[k]) continue;                // (what was read there may be NaN)
      float f[KE];
      DL::unpack(vr[k], f);
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        const float pk = s[k][h] == -INFINITY ? 0.f : exp2f(s[k][h] - m[h]);
        l[h] += pk;
        const float pw = BLK ? pk * vs[k] : pk;
        if constexpr (kPairs) {
          const uint64_t p2 = f2pack(pw, pw);
#pragma unroll
          for (int e = 0; e < KE; e += 2)
            f2unpack(ffma2(p2, f2pack(f[e], f[e + 1]), f2pack(o[h][e], o[h][e + 1])), o[h][e], o[h][e + 1]);
        } else {
#pragma unroll
          for (int e = 0; e < KE; ++e) o[h][e] = fmaf(pw, f[e], o[h][e]);
        }
      }
    }
  }
  // lane groups of a warp (equal li: equal dims), then the warps
#pragma unroll
  for (int off = LPT; off < 32; off <<= 1) {
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[h], off), l2 = __shfl_xor_sync(0xffffffffu, l[h], off);
      const float M = fmaxf(m[h], m2);
      const float a = m[h] == -INFINITY ? 0.f : exp2f(m[h] - M), c = m2 == -INFINITY ? 0.f : exp2f(m2 - M);
      l[h] = a * l[h] + c * l2;
#pragma unroll
      for (int e = 0; e < KE; ++e) {
        const float o2 = __shfl_xor_sync(0xffffffffu, o[h][e], off);
        o[h][e] = a * o[h][e] + c * o2;
      }
      m[h] = M;
    }
  }
  if (grp == 0) {
#pragma unroll
    for (int h = 0; h < GT; ++h) {
#pragma unroll
      for (int e = 0; e < KE; ++e) so[warp][h][li * KE + e] = o[h][e];
      if (li == 0) {
        sm[warp][h] = m[h];
        sl[warp][h] = l[h];
      }
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < gh * D; x += kDirectWarps * 32) {
    const int h = x / D, d = x % D;
    float M = sm[0][h];
#pragma unroll
    for (int w = 1; w < kDirectWarps; ++w) M = fmaxf(M, sm[w][h]);
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kDirectWarps; ++w) {
      const float a = sm[w][h] == -INFINITY ? 0.f : exp2f(sm[w][h] - M);
      num = fmaf(a, so[w][h][d], num);
      den = fmaf(a, sl[w][h], den);
    }
    const size_t bh = (size_t)b * p.Hq + h0 + h;
    const size_t slot = bh * p.max_parts + part;
    if (nparts > 1) p.ws_o[slot * D + d] = num;
    else E::store1(static_cast<T*>(p.out) + bh * D + d, den != 0.f ? num / den : 0.f);
    if (d == 0 && (W || nparts > 1)) {
      p.ws_ml[slot * 2] = M;
      p.ws_ml[slot * 2 + 1] = den;
    }
  }
}

}  // namespace
}  // namespace pa
