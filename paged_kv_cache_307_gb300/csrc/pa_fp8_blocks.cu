// pa_fp8_blocks.cu — quantising append into an e4m3 pool with one power-of-two
// scale per (block, KV head).
//
// For every block that a sequence's new tokens touch and every head, K and V
// apart:
//   a    = max |x| over the block's new finite elements of the head
//   need = the smallest power of two with a <= 448 * need (at least 2^-100; 0 when a is 0)
//   s    = max(need, the block's scale if it holds earlier tokens of the sequence)
//   new codes = e4m3(x / s), saturating; earlier codes c become e4m3(value(c) * old / s)
// A power of two costs a floating-point code nothing: its relative precision
// is the same at every exponent, x / s is exact, and raising the scale of codes
// written before shifts their exponents, which is exact but for values that
// fall below the smallest normal code.  So a block filled token by token holds
// what one filled at once holds, up to those.
//
// One warp per (touched block, head): the block's new rows of the head, K's and V's,
// 16 bytes per lane, stay in registers from the maximum to the codes as far as 16
// chunks a lane reach (sixteen loads in flight: all of a bf16 block of 16 x 128); of
// larger blocks (f32, or 32 tokens) the rest is read a second time, out of the caches.
// Blocks are owned by one warp each, so nothing is atomic.  Which block a warp works on
// needs no scan over the sequences: sequence b's units start at
//   U_b = floor(query_start[b] / bs) + 2 b,
// and n tokens touch at most floor((n - 1) / bs) + 2 blocks, which never passes
// U_{b+1}; a search over query_start finds b, and surplus units leave.
// Bound by HBM: reads elem and writes 1 byte per element.  A warp's life is a chain of
// five latencies (starts, length, block id, rows, and the writes), so what counts is the
// bytes that an SM's warps have in flight, then the instructions per element: 8 prompts
// of 3000 to 4096 tokens x 8 heads x 128 in bf16 (174 MB in all) take 34.8 us (5.0 TB/s,
// 74 % of the copy rate) with K and V in one warp at four CTAs of 128 registers per SM
// and 41 at five; 37.0 with the maximum taken over floats and not over their bits, and
// so 41 and 44 at three and five CTAs, and with a warp for K and one for V 43, 38 and 45
// at three, six and eight.  One token for 64 sequences x 32 heads takes 7 us on the GPU,
// launch and latencies.
#include "pa_common.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_fp8_blocks;

constexpr int kWarps = 4;
constexpr int kHeld = 8;               // 16-byte chunks a lane keeps
constexpr float kMinScale = 7.888609052210118e-31f;   // 2^-100
constexpr float kE4m3Max = 448.f;

// The smallest power of two s with a <= 448 s, not below 2^-100; 0 for 0.
// (448 = 1.75 * 2^8: a = m * 2^e with m in [1, 2) needs 2^(e-8), or 2^(e-7) when m > 1.75.)
__device__ __forceinline__ float pow2_scale(float a) {
  if (!(a > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 127;                 // a subnormal counts as 2^-127: the floor applies
  const int k = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return k < -100 ? kMinScale : __uint_as_float((uint32_t)(k + 127) << 23);
}

// Magnitudes of 16 bytes of elements as integers, ordered like the values.
template <typename T> struct Magnitude;
template <> struct Magnitude<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f80u;
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // the running maxima of the even and the odd elements, with those of x
  __device__ __forceinline__ static uint32_t top(const uint4& x, uint32_t m) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    return max2(max2(max2(m, x.x & kAbs), max2(x.y & kAbs, x.z & kAbs)), x.w & kAbs);
  }
  __device__ __forceinline__ static uint32_t one(uint32_t m) { return max(m & 0xffffu, m >> 16); }
  __device__ __forceinline__ static uint32_t finite_top(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = w[k] & 0x7fffu, b = (w[k] >> 16) & 0x7fffu;
      m = max(m, max(a < kInf ? a : 0u, b < kInf ? b : 0u));
    }
    return m;
  }
  __device__ __forceinline__ static float value(uint32_t m) { return __uint_as_float(m << 16); }
};
template <> struct Magnitude<float> {
  static constexpr uint32_t kInf = 0x7f800000u, kAbs = 0x7fffffffu;
  __device__ __forceinline__ static uint32_t top(const uint4& x, uint32_t m) {
    return max(max(max(m, x.x & kAbs), max(x.y & kAbs, x.z & kAbs)), x.w & kAbs);
  }
  __device__ __forceinline__ static uint32_t one(uint32_t m) { return m; }
  __device__ __forceinline__ static uint32_t finite_top(const uint4& x) {
    const uint32_t w[4] = {x.x & kAbs, x.y & kAbs, x.z & kAbs, x.w & kAbs};
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, w[k] < kInf ? w[k] : 0u);
    return m;
  }
  __device__ __forceinline__ static float value(uint32_t m) { return __uint_as_float(m); }
};

// Two conversions of two values each, the first value in the low byte.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

struct AppendParams {
  const void* src[2];            // key, value [T, Hkv, D]
  uint8_t* pool[2];
  float* scale[2];
  const int32_t* query_start;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int B, T, Hkv, D, bs, max_blocks, num_blocks, scale_row;
};

// Whether sequence b's rows lie in [0, T] and its new tokens in its context, and
// the context in its table row.
__device__ __forceinline__ bool good_seq(const AppendParams& p, int b) {
  const int s0 = __ldg(&p.query_start[b]), s1 = __ldg(&p.query_start[b + 1]);
  const int L = __ldg(&p.context_lens[b]);
  return s0 >= 0 && s1 >= s0 && s1 <= p.T && L >= 0 && L <= p.max_blocks * p.bs && s1 - s0 <= L;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 4) append_kernel(const AppendParams p) {
  using E = Elem<T>;
  using M = Magnitude<T>;
  constexpr int EPC = E::kPerChunk;
  const int lane = threadIdx.x & 31;
  const int h = (int)blockIdx.y * kWarps + (int)(threadIdx.x >> 5);
  const int u = (int)blockIdx.x;
  if (u == 0 && blockIdx.y == 0) {
    // every sequence's arguments are looked at once, whatever units it has
    for (int i = (int)threadIdx.x; i < p.B; i += kWarps * 32)
      if (!good_seq(p, i)) atomicOr(&g_status_fp8_blocks, PA_DEV_BAD_LEN);
  }
  const int b = find_unit(p.query_start, p.B, p.bs, 2, u);
  const int s0 = __ldg(&p.query_start[b]), s1 = __ldg(&p.query_start[b + 1]);
  const int L = __ldg(&p.context_lens[b]);
  const int i = u - (s0 / p.bs + 2 * b);        // the sequence's i-th touched block
  const int n = s1 - s0;
  if (!good_seq(p, b)) return;
  if (n == 0 || i < 0 || h >= p.Hkv) return;
  const int j = (L - n) / p.bs + i;             // logical block
  if (j >= (L + p.bs - 1) / p.bs) return;
  const int blk = __ldg(&p.block_tables[(size_t)b * p.max_blocks + j]);
  if ((unsigned)blk >= (unsigned)p.num_blocks) {
    if (h == 0 && lane == 0) atomicOr(&g_status_fp8_blocks, PA_DEV_BAD_BLOCK);
    return;
  }
  const int first = max(L - n - j * p.bs, 0);   // the block's first new slot; earlier ones hold tokens
  const int cnt = min(L - j * p.bs, p.bs) - first;
  const size_t row = (size_t)p.Hkv * p.D;       // elements from token to token, in the source and in the pool
  const size_t from = ((size_t)(s0 + j * p.bs + first - (L - n)) * row + (size_t)h * p.D) * sizeof(T);
  const size_t to = (size_t)blk * p.bs * row + (size_t)h * p.D;
  const size_t sat = (size_t)blk * p.scale_row + h;
  const int csh = 31 - __clz(p.D / EPC), cpr = 1 << csh;   // 16-byte source chunks per row: 4, 8, 16 or 32
  const int chunks = cnt << csh;
  auto fetch = [&](int kv, int c) {
    return ld_nc_v4(static_cast<const unsigned char*>(p.src[kv]) + from +
                    ((size_t)(c >> csh) * row + (size_t)(c & (cpr - 1)) * EPC) * sizeof(T));
  };
  // K's and V's first kHeld chunks per lane stay in registers from the maximum to the
  // codes (all of a bf16 block of 16 x 128), the rest is read again
  uint4 held[2][kHeld];
  float olds[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      held[kv][k] = lane + 32 * k < chunks ? fetch(kv, lane + 32 * k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) olds[kv] = first > 0 ? p.scale[kv][sat] : 0.f;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    // the largest magnitude, by its bits; elements that are not finite are above all others
    // and leave the maximum to a second look at the finite ones
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) top = M::top(held[kv][k], top);
#pragma unroll 4
    for (int c = lane + 32 * kHeld; c < chunks; c += 32) top = M::top(fetch(kv, c), top);
    top = __reduce_max_sync(0xffffffffu, M::one(top));
    if (top >= M::kInf) {
      top = 0u;
      for (int c = lane; c < chunks; c += 32) top = max(top, M::finite_top(fetch(kv, c)));
      top = __reduce_max_sync(0xffffffffu, top);
    }
    const float amax = M::value(top);
    const float old = olds[kv];
    const float s = fmaxf(old, pow2_scale(amax));
    const float inv = s > 0.f ? 1.f / s : 0.f;    // exact: s is a power of two
    __syncwarp();
    if (lane == 0 && (first == 0 || s != old)) p.scale[kv][sat] = s;
    uint8_t* dst = p.pool[kv] + to;
    if (first > 0 && s > old) {
      // the earlier tokens' codes under the raised scale, 16 codes per lane
      const float f = old * inv;
      const int c16 = p.D / 16;
      for (int c = lane; c < first * c16; c += 32) {
        uint8_t* at = dst + (size_t)(c / c16) * row + (size_t)(c % c16) * 16;
        float v[16];
        Elem<fp8e4m3>::unpack(*reinterpret_cast<const uint4*>(at), v);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= f;
        st_v4(at, make_uint4(encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7]),
                             encode4(v[8], v[9], v[10], v[11]), encode4(v[12], v[13], v[14], v[15])));
      }
    }
    dst += (size_t)first * row;
    auto put = [&](int c, const uint4& x) {
      float f[EPC];
      E::unpack(x, f);
      uint32_t w[EPC / 4];
#pragma unroll
      for (int k = 0; k < EPC / 4; ++k)
        w[k] = encode4(f[4 * k] * inv, f[4 * k + 1] * inv, f[4 * k + 2] * inv, f[4 * k + 3] * inv);
      uint8_t* at = dst + (size_t)(c >> csh) * row + (size_t)(c & (cpr - 1)) * EPC;
      if constexpr (EPC == 8) {
        *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t*>(at) = w[0];
      }
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (lane + 32 * k < chunks) put(lane + 32 * k, held[kv][k]);
#pragma unroll 4
    for (int c = lane + 32 * kHeld; c < chunks; c += 32) put(c, fetch(kv, c));
  }
}

}  // namespace

unsigned* status_word_fp8_blocks() { return device_word(g_status_fp8_blocks); }

}  // namespace pa

using namespace pa;

extern "C" int pa_append_fp8_blocks(const void* key, const void* value, const int32_t* query_start,
                                    int total_tokens, const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* context_lens, int num_seqs, void* k_cache, void* v_cache,
                                    float* k_scale, float* v_scale, int num_blocks, int block_size,
                                    int num_kv_heads, int head_dim, pa_dtype src_dtype, void* stream) {
  if (src_dtype != PA_F32 && src_dtype != PA_BF16) return PA_ERR_DTYPE;
  if (total_tokens < 0 || num_seqs < 0 || num_blocks <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
      !supported_head_dim(head_dim) || !supported_block_size(block_size))
    return PA_ERR_SHAPE;
  if ((long long)max_blocks_per_seq * block_size > kMaxRowTokens ||
      (long long)total_tokens / block_size + 2ll * num_seqs > 0x3fffffffll)
    return PA_ERR_SHAPE;
  const long long groups = ((long long)num_kv_heads + kWarps - 1) / kWarps;
  if (groups > 65535) return PA_ERR_SHAPE;
  if (total_tokens == 0 || num_seqs == 0) return PA_OK;
  if (!key || !value || !query_start || !block_tables || !context_lens || !k_cache || !v_cache || !k_scale || !v_scale)
    return PA_ERR_NULL;
  if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
      !aligned16(v_scale))
    return PA_ERR_ALIGN;
  AppendParams p;
  p.src[0] = key;
  p.src[1] = value;
  p.pool[0] = static_cast<uint8_t*>(k_cache);
  p.pool[1] = static_cast<uint8_t*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.B = num_seqs;
  p.T = total_tokens;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  p.bs = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.scale_row = scale_row(num_kv_heads);
  const dim3 grid((unsigned)(total_tokens / block_size + 2 * num_seqs), (unsigned)groups);
  if (src_dtype == PA_BF16)
    append_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else
    append_kernel<float><<<grid, kWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return ck(cudaGetLastError(), "launch append_kernel") ? PA_OK : PA_ERR_CUDA;
}
