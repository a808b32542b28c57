// pa_rope.cu — rotary positions: queries and keys rotated, the keys on their way into a
// paged cache (pa_rope, pa_rope_and_cache) or, as the one key that all heads share, into a
// latent cache (pa_latent_append).
//
// Pair i of a head at position p turns by the angle p f_i:
//   (x, y) -> A (x cos - y sin, y cos + x sin)
// The angle is never formed.  The caller's table holds f_i / 2 pi as a 64-bit fraction of a
// turn, and p times that, modulo 2^64, is the turn's fraction exactly: the integer product
// wraps where an angle would have to be reduced.  (An fp32 angle is off by 2^-24 of itself,
// 0.06 at a position of a million.)  The fraction as a float goes to sincospif.
//
// Data movement bound by HBM: every element is read and written once, in 16-byte chunks.
// A CTA takes p.tpb tokens; their cosines and sines are made once, in shared memory, for
// all heads.  A work unit is what one pass over registers needs: in the half layout two
// chunks, half the rotated part apart; else one chunk.  A thread keeps its unit of a token
// and walks the tokens: what the unit is costs it two divisions in all (found anew for every
// token, they took 8192 tokens of 40 heads x 128 from 31 to 38 us, 64 tokens of a step from 2.9
// to 4.2; what is left bounds it still: the issue slots are 0.7 full).
#include "pa_common.cuh"
#include "pa_mma.cuh"

#include <math.h>

namespace pa {
namespace {

__device__ unsigned g_status_rope;

constexpr int kThreads = 256;
// Tokens a CTA takes side by side with as many as its threads have in flight: four, or two twice in
// the half layout, whose units are twice as large; and CTAs an SM.  8192 tokens of 40 heads x 128,
// interleaved, take 28.7 us (5.8 TB/s); two in flight 36, six CTAs 33, four 40.  5000 tokens of 20
// heads x 64 in f32, half layout, take 8.9 us (5.8 TB/s); four in flight 13, six CTAs 9.7.
constexpr int kTokens = 4;
constexpr int kMinCtas = 5;
constexpr int kTableEntries = 2048;      // (cos, sin) pairs in shared memory

// One tensor of rows: bytes from token to token and head to head.
struct Part {
  const char* src;
  char* dst;
  long long src_token, src_head, dst_token, dst_head;
  int units;                             // of a head
  int all;                               // of a token
  uint32_t per;                          // 2^32 / units, rounded up: r / units is the upper word of r * per
};

struct RopeParams {
  Part q, k, c;                          // rotated; rotated (by slot where slots is given); copied by slot
  const int32_t* positions;
  const int64_t* slots;
  const uint64_t* steps;
  long long num_slots;
  float amplitude;
  int n, tpb, items;                     // tokens, tokens a CTA, units a token
  int pairs;                             // rotated pairs of a head
  uint32_t per_pairs;                    // likewise
};

__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float* f) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// HALF: pair i is elements i and pairs + i of a head; else 2i and 2i + 1.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, kMinCtas) rope_kernel(const RopeParams p) {
  using E = Elem<T>;
  constexpr int EPC = E::kPerChunk;
  constexpr int kPairs = HALF ? EPC : EPC / 2;             // pairs of a unit
  constexpr int kBatch = HALF ? kTokens / 2 : kTokens;     // tokens in flight per thread
  __shared__ __align__(16) float2 table[kTableEntries];
  const int tok0 = blockIdx.x * p.tpb;
  const int nt = min(p.tpb, p.n - tok0);
  const int hop = p.pairs * E::kBytes;                     // HALF: from a pair's first element to its second

  // ---- the thread's units: tokens with few units share the CTA side by side
  const int side = p.items < kThreads ? kThreads / p.items : 1;
  int sub = 0, r0 = (int)(blockIdx.y * kThreads + threadIdx.x);
  if (side > 1) {
    sub = (int)threadIdx.x / p.items;
    r0 = sub < side ? (int)threadIdx.x - sub * p.items : p.items;
  }
  const int turned = p.pairs / kPairs;                     // units of a head that are rotated

  const char* src = nullptr;                               // the unit's bytes of token tok0
  char* dst = nullptr;
  long long src_token = 0, dst_token = 0;
  int x = 0;
  bool turn = false, by_slot = false, first = false;
  auto unit = [&](int r) {
    const bool is_q = r < p.q.all, is_c = !is_q && r >= p.q.all + p.k.all;
    r -= is_q ? 0 : is_c ? p.q.all + p.k.all : p.q.all;
    const uint32_t per = is_q ? p.q.per : is_c ? p.c.per : p.k.per;
    const int units = is_q ? p.q.units : is_c ? p.c.units : p.k.units;
    const int h = units > 1 ? (int)__umulhi((uint32_t)r, per) : r;
    x = r - h * units;
    turn = !is_c && x < turned;
    by_slot = !is_q && p.slots;
    first = !is_c && r == 0;
    const int off = x * 16 + (HALF && !is_c && !turn ? turned * 16 : 0);    // (each rotated unit was two chunks)
    src_token = is_q ? p.q.src_token : is_c ? p.c.src_token : p.k.src_token;
    dst_token = is_q ? p.q.dst_token : is_c ? p.c.dst_token : p.k.dst_token;
    src = (is_q ? p.q.src : is_c ? p.c.src : p.k.src) + tok0 * src_token +
          h * (is_q ? p.q.src_head : is_c ? p.c.src_head : p.k.src_head) + off;
    dst = (is_q ? p.q.dst : is_c ? p.c.dst : p.k.dst) + h * (is_q ? p.q.dst_head : is_c ? p.c.dst_head : p.k.dst_head) + off;
  };

  char* d[kBatch];                                         // null: nothing to do
  uint4 lo[kBatch], hi[kBatch];
  auto load = [&](int t) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b, t += side) {
      d[b] = nullptr;
      if (t >= nt) continue;
      long long row = tok0 + t;
      if (by_slot) {
        row = __ldg(reinterpret_cast<const long long*>(p.slots) + row);
        if (row < 0) continue;                             // padding
        if (row >= p.num_slots) {
          if (first) atomicOr(&g_status_rope, PA_DEV_BAD_SLOT);
          continue;
        }
      }
      const char* s = src + t * src_token;
      d[b] = dst + row * dst_token;
      lo[b] = ld_v4(s);
      if (HALF && turn) hi[b] = ld_v4(s + hop);
    }
  };
  auto finish = [&](int t) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b, t += side) {
      if (!d[b]) continue;
      if (!turn) {
        st_v4(d[b], lo[b]);
        continue;
      }
      const float4* cs = reinterpret_cast<const float4*>(table + t * p.pairs + x * kPairs);
      float v[EPC], w[EPC];
      E::unpack(lo[b], v);
      if constexpr (HALF) {
        E::unpack(hi[b], w);
#pragma unroll
        for (int e = 0; e < EPC; e += 2) {
          const float4 f = cs[e / 2];                      // cos, sin of two pairs
          const float v0 = v[e], v1 = v[e + 1];
          v[e] = fmaf(v0, f.x, -w[e] * f.y);
          w[e] = fmaf(w[e], f.x, v0 * f.y);
          v[e + 1] = fmaf(v1, f.z, -w[e + 1] * f.w);
          w[e + 1] = fmaf(w[e + 1], f.z, v1 * f.w);
        }
        st_v4(d[b] + hop, pack<T>(w));
        st_v4(d[b], pack<T>(v));
      } else {
#pragma unroll
        for (int e = 0; e < EPC; e += 4) {
          const float4 f = cs[e / 4];
          w[e] = fmaf(v[e], f.x, -v[e + 1] * f.y);
          w[e + 1] = fmaf(v[e + 1], f.x, v[e] * f.y);
          w[e + 2] = fmaf(v[e + 2], f.z, -v[e + 3] * f.w);
          w[e + 3] = fmaf(v[e + 3], f.z, v[e + 2] * f.w);
        }
        st_v4(d[b], pack<T>(w));
      }
    }
  };

  if (r0 < p.items) {                                      // (on its way while the table is made)
    unit(r0);
    load(sub);
  }
  for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
    const int t = (int)__umulhi((uint32_t)i, p.per_pairs);
    const uint64_t phase = (uint64_t)(int64_t)__ldg(&p.positions[tok0 + t]) * __ldg(&p.steps[i - t * p.pairs]);
    // the turn's fraction in [-1/2, 1/2), in half turns (its upper word: 2^-33 of a turn)
    float sn, cn;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn, &cn);
    table[i] = make_float2(cn * p.amplitude, sn * p.amplitude);
  }
  __syncthreads();
  for (int r = r0; r < p.items;) {
    for (int t = sub;;) {
      finish(t);
      t += kBatch * side;
      if (t >= nt) break;
      load(t);
    }
    r += (int)gridDim.y * kThreads;
    if (side > 1 || r >= p.items) break;
    unit(r);
    load(sub);
  }
}

// ---------------------------------------------------------------------------- host
// A sum of two doubles, 106 bits: a step needs 64, of which a position of 2^31 leaves 33.  (In 53 bits
// a step was off by up to 350 units, 2^-24 of a turn at that position.)
struct Twice {
  double hi, lo;
};
Twice sum(double a, double b) {              // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
Twice mul(Twice a, Twice b) {
  const double p = a.hi * b.hi;
  return sum(p, fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p))));
}
Twice div(Twice a, double b) {
  const double q = a.hi / b;
  return sum(q, (fma(-q, b, a.hi) + a.lo) / b);
}
// 1 - a
Twice less(Twice a) {
  const Twice d = sum(1.0, -a.hi);           // (0 <= a <= 1)
  return sum(d.hi, d.lo - a.lo);
}
// x^(-1/n): one step of Newton's method from the double next to it leaves an error of about 2^-95.
Twice inverse_root(double x, int n) {
  const double r = pow(x, -1.0 / n);
  Twice p{x, 0.0};
  for (int i = 0; i < n; ++i) p = mul(p, Twice{r, 0.0});
  return sum(r, r * (((1.0 - p.hi) - p.lo) / n));
}

struct Rows {                            // a strided [tokens, heads, dim] tensor, strides in elements
  const void* data;
  long long token, head;
};

bool aligned_rows(const Rows& r, int e) {
  return aligned16(r.data) && (r.token * e) % 16 == 0 && (r.head * e) % 16 == 0;
}

// A rotated part; what lies behind the rotated elements moves along unless it is in place already.
Part turned_part(const Rows& dst, const Rows& src, int heads, int dim, int rot, int e, bool half, bool by_slot) {
  Part a = {};
  a.src = static_cast<const char*>(src.data);
  a.dst = static_cast<char*>(const_cast<void*>(dst.data));
  a.src_token = src.token * e;
  a.src_head = src.head * e;
  a.dst_token = dst.token * e;
  a.dst_head = dst.head * e;
  const bool in_place = !by_slot && dst.data == src.data && dst.token == src.token && dst.head == src.head;
  a.units = rot * e / (half ? 32 : 16) + (in_place ? 0 : (dim - rot) * e / 16);
  a.all = heads * a.units;
  return a;
}

Part copied_part(void* dst, long long dst_row, const Rows& src, int heads, int dim, int e) {
  Part a = {};
  a.src = static_cast<const char*>(src.data);
  a.dst = static_cast<char*>(dst);
  a.src_token = src.token * e;
  a.src_head = src.head * e;
  a.dst_token = dst_row * e;
  a.dst_head = (long long)dim * e;
  a.units = dim * e / 16;
  a.all = heads * a.units;
  return a;
}

// (a token's units then fit 32 bits)
bool heads_in_range(int n) { return n >= 0 && n <= 1 << 20; }

bool rotary_shape(int dim, int rot) { return rot > 0 && rot <= dim && rot % 16 == 0 && dim % 16 == 0 && dim <= 512; }

int launch(RopeParams& p, pa_dtype dtype, bool half, void* stream) {
  const long long items = (long long)p.q.all + p.k.all + p.c.all;
  if (items > 1 << 24) return PA_ERR_SHAPE;
  if (items == 0) return PA_OK;
  p.items = (int)items;
  auto per = [](int n) { return n > 1 ? (uint32_t)(((1ull << 32) + n - 1) / n) : 0u; };
  for (Part* a : {&p.q, &p.k, &p.c}) {
    if (a->units == 0) a->units = 1;
    a->per = per(a->units);
  }
  p.per_pairs = per(p.pairs);
  // Tokens a CTA, as far as shared memory holds their cosines and the GPU gets four CTAs an SM; the
  // units of few tokens are divided among CTAs as well.
  const int side = items < kThreads ? (int)(kThreads / items) : 1;
  const int most = kTableEntries / p.pairs;
  const long long spread = (long long)p.n / (4 * kTunedSms);
  long long tpb = spread < most ? spread : most;
  tpb = tpb < kTokens * side ? tpb : kTokens * side;
  p.tpb = (int)(tpb < 1 ? 1 : tpb);
  const unsigned grid = (unsigned)((p.n + (long long)p.tpb - 1) / p.tpb);
  const long long all = (items + kThreads - 1) / kThreads, room = 8ll * kTunedSms / grid;
  const unsigned groups = (unsigned)(all < room ? all : room < 1 ? 1 : room < 65535 ? room : 65535);
  auto kernel = dtype == PA_F32 ? (half ? &rope_kernel<float, true> : &rope_kernel<float, false>)
                                : (half ? &rope_kernel<__nv_bfloat16, true> : &rope_kernel<__nv_bfloat16, false>);
  void* args[] = {&p};
  return ck(cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid, groups), dim3(kThreads), args, 0,
                             (cudaStream_t)stream),
            "cudaLaunchKernel(rope_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

unsigned* status_word_rope() { return device_word(g_status_rope); }

}  // namespace pa

using namespace pa;

extern "C" int pa_rope_steps(uint64_t* steps, float* amplitude, int rotary_dim, double base, pa_rope_scaling scaling,
                             double factor, double original_len, double beta_fast, double beta_slow) {
  constexpr double kPi = 3.14159265358979323846;
  if (rotary_dim <= 0 || rotary_dim % 16 || rotary_dim > 512 || !(base > 1.0) || !(base < 1e300)) return PA_ERR_SHAPE;
  if (scaling < PA_ROPE_PLAIN || scaling > PA_ROPE_YARN) return PA_ERR_SHAPE;
  if (scaling != PA_ROPE_PLAIN && !(factor >= 1.0 && factor < 1e30)) return PA_ERR_SHAPE;
  if (scaling == PA_ROPE_YARN && !(original_len > 0.0 && original_len < 1e30 && beta_slow > 0.0 && beta_fast >= beta_slow && beta_fast < 1e30))
    return PA_ERR_SHAPE;
  if (!steps || !amplitude) return PA_ERR_NULL;
  const double d = rotary_dim;
  double lo = 0.0, hi = 0.0;
  if (scaling == PA_ROPE_YARN) {
    auto pair = [&](double turns) { return d * log(original_len / (turns * 2.0 * kPi)) / (2.0 * log(base)); };
    lo = fmax(0.0, floor(pair(beta_fast)));
    hi = fmin(d - 1.0, ceil(pair(beta_slow)));
  }
  // f_i = ratio^i; the raised base's is base^(-2 i / d) factor^(-2 i / (d - 2))
  Twice ratio = inverse_root(base, rotary_dim / 2);
  if (scaling == PA_ROPE_NTK) ratio = mul(ratio, inverse_root(factor, rotary_dim / 2 - 1));
  const Twice kTurn{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / 2 pi
  Twice f{1.0, 0.0};
  for (int i = 0; i < rotary_dim / 2; ++i, f = mul(f, ratio)) {
    Twice t = mul(f, kTurn);
    if (scaling == PA_ROPE_LINEAR) t = div(t, factor);
    if (scaling == PA_ROPE_YARN) {
      // 1 - part (1 - 1 / factor)
      const double n = hi - lo < 1e-3 ? 1e-3 : hi - lo;
      const Twice part = i <= lo ? Twice{0.0, 0.0} : i - lo >= n ? Twice{1.0, 0.0} : div(Twice{i - lo, 0.0}, n);
      t = mul(t, less(mul(part, less(div(Twice{1.0, 0.0}, factor)))));
    }
    // the nearest whole number of 2^-64 turns
    const double whole = floor(ldexp(t.hi, 64));
    steps[i] = (uint64_t)whole + (uint64_t)(int64_t)floor((ldexp(t.hi, 64) - whole) + ldexp(t.lo, 64) + 0.5);
  }
  *amplitude = scaling == PA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return PA_OK;
}

extern "C" int pa_rope(void* q_out, long long q_out_token_stride, long long q_out_head_stride, const void* q,
                       long long q_token_stride, long long q_head_stride, int num_heads, void* k_out,
                       long long k_out_token_stride, long long k_out_head_stride, const void* k,
                       long long k_token_stride, long long k_head_stride, int num_kv_heads,
                       const int32_t* positions, int num_tokens, int head_dim, int rotary_dim, pa_rope_layout layout,
                       const uint64_t* steps, float amplitude, pa_dtype dtype, void* stream) {
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (num_tokens < 0 || !heads_in_range(num_heads) || !heads_in_range(num_kv_heads) || !rotary_shape(head_dim, rotary_dim) ||
      (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED))
    return PA_ERR_SHAPE;
  if (num_tokens == 0 || (num_heads == 0 && num_kv_heads == 0)) return PA_OK;
  if ((num_heads && (!q || !q_out)) || (num_kv_heads && (!k || !k_out)) || !positions || !steps) return PA_ERR_NULL;
  const int e = elem_bytes(dtype);
  const Rows qs{q, q_token_stride, q_head_stride}, qd{q_out, q_out_token_stride, q_out_head_stride};
  const Rows ks{k, k_token_stride, k_head_stride}, kd{k_out, k_out_token_stride, k_out_head_stride};
  if ((num_heads && (!aligned_rows(qs, e) || !aligned_rows(qd, e))) ||
      (num_kv_heads && (!aligned_rows(ks, e) || !aligned_rows(kd, e))))
    return PA_ERR_ALIGN;
  const bool half = layout == PA_ROPE_HALF;
  RopeParams p = {};
  if (num_heads) p.q = turned_part(qd, qs, num_heads, head_dim, rotary_dim, e, half, false);
  if (num_kv_heads) p.k = turned_part(kd, ks, num_kv_heads, head_dim, rotary_dim, e, half, false);
  p.positions = positions;
  p.steps = steps;
  p.amplitude = amplitude;
  p.n = num_tokens;
  p.pairs = rotary_dim / 2;
  return launch(p, dtype, half, stream);
}

extern "C" int pa_rope_and_cache(void* q_out, long long q_out_token_stride, long long q_out_head_stride,
                                 const void* q, long long q_token_stride, long long q_head_stride, int num_heads,
                                 const void* key, long long key_token_stride, long long key_head_stride,
                                 const void* value, long long value_token_stride, long long value_head_stride,
                                 int num_kv_heads, const int32_t* positions, const int64_t* slot_mapping,
                                 int num_tokens, void* k_cache, void* v_cache, int num_blocks, int block_size,
                                 int head_dim, int rotary_dim, pa_rope_layout layout, const uint64_t* steps,
                                 float amplitude, pa_dtype dtype, void* stream) {
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (num_tokens < 0 || !heads_in_range(num_heads) || !heads_in_range(num_kv_heads) || num_kv_heads == 0 || num_blocks <= 0 || !supported_head_dim(head_dim) ||
      !supported_block_size(block_size) || !rotary_shape(head_dim, rotary_dim) ||
      (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED))
    return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if ((num_heads && (!q || !q_out)) || !key || !value || !positions || !slot_mapping || !k_cache || !v_cache || !steps)
    return PA_ERR_NULL;
  const int e = elem_bytes(dtype);
  const Rows qs{q, q_token_stride, q_head_stride}, qd{q_out, q_out_token_stride, q_out_head_stride};
  const Rows ks{key, key_token_stride, key_head_stride}, vs{value, value_token_stride, value_head_stride};
  const long long row = (long long)num_kv_heads * head_dim;
  const Rows kd{k_cache, row, head_dim};
  if ((num_heads && (!aligned_rows(qs, e) || !aligned_rows(qd, e))) || !aligned_rows(ks, e) || !aligned_rows(vs, e) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_ALIGN;
  const bool half = layout == PA_ROPE_HALF;
  RopeParams p = {};
  if (num_heads) p.q = turned_part(qd, qs, num_heads, head_dim, rotary_dim, e, half, false);
  p.k = turned_part(kd, ks, num_kv_heads, head_dim, rotary_dim, e, half, true);
  p.c = copied_part(v_cache, row, vs, num_kv_heads, head_dim, e);
  p.positions = positions;
  p.slots = slot_mapping;
  p.num_slots = (long long)num_blocks * block_size;
  p.steps = steps;
  p.amplitude = amplitude;
  p.n = num_tokens;
  p.pairs = rotary_dim / 2;
  return launch(p, dtype, half, stream);
}

extern "C" int pa_latent_append(const void* latent, long long latent_stride, const void* key_rope,
                                long long key_rope_stride, void* query_out, long long query_out_token_stride,
                                long long query_out_head_stride, const void* query, long long query_token_stride,
                                long long query_head_stride, int num_heads, const int32_t* positions,
                                const int64_t* slot_mapping, int num_tokens, void* cache, int num_blocks,
                                int block_size, int latent_dim, int rope_dim, pa_rope_layout layout,
                                const uint64_t* steps, float amplitude, pa_dtype dtype, void* stream) {
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (num_tokens < 0 || !heads_in_range(num_heads) || num_blocks <= 0 || !latent_shape(latent_dim, rope_dim, block_size) ||
      (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED))
    return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!latent || !key_rope || (num_heads && (!query || !query_out)) || !positions || !slot_mapping || !cache || !steps)
    return PA_ERR_NULL;
  const int e = elem_bytes(dtype);
  const long long row = latent_dim + rope_dim;
  const Rows ls{latent, latent_stride, 0}, ks{key_rope, key_rope_stride, 0};
  const Rows qs{query, query_token_stride, query_head_stride};
  const Rows qd{query_out, query_out_token_stride, query_out_head_stride};
  if (!aligned_rows(ls, e) || !aligned_rows(ks, e) || !aligned16(cache) ||
      (num_heads && (!aligned_rows(qs, e) || !aligned_rows(qd, e))))
    return PA_ERR_ALIGN;
  const bool half = layout == PA_ROPE_HALF;
  RopeParams p = {};
  if (num_heads) p.q = turned_part(qd, qs, num_heads, rope_dim, rope_dim, e, half, false);
  const Rows kd{static_cast<char*>(cache) + (size_t)latent_dim * e, row, 0};
  p.k = turned_part(kd, ks, 1, rope_dim, rope_dim, e, half, true);
  p.c = copied_part(cache, row, ls, 1, latent_dim, e);
  p.positions = positions;
  p.slots = slot_mapping;
  p.num_slots = (long long)num_blocks * block_size;
  p.steps = steps;
  p.amplitude = amplitude;
  p.n = num_tokens;
  p.pairs = rope_dim / 2;
  return launch(p, dtype, half, stream);
}
