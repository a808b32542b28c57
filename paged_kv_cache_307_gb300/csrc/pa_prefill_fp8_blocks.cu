// pa_prefill_fp8_blocks.cu — causal attention of each sequence's newest tokens
// over an e4m3 pool with one scale per (block, KV head).
//
// Row i of sequence b (n_b rows, the last n_b tokens of its context) sits at
// position p = L_b - n_b + i and attends to the keys at 0..p:
//   out = sum_t softmax_t(scale * <q, K_t>) V_t,  K = value(code) * k_scale[block, head], V likewise.
//
// rows_kernel: one warp per (row, query head), any sizes.  Lane t of a step of
// 32 keys computes one key's whole score from its row of codes; the warp takes
// the running maximum and sum, then every lane accumulates its D / 32 head
// dims over the 32 keys.  The block's K scale multiplies the score, its V scale
// the softmax weight; the sum of the softmax is over the unscaled weights.
#include "pa_common.cuh"

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
  int lo = 0, hi = p.B - 1;                    // the last sequence that starts at or before the row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(&p.query_start[mid]) <= row) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo;
  if (!good_rows(p, b)) return;
  const int r0 = __ldg(&p.query_start[b]), r1 = __ldg(&p.query_start[b + 1]);
  if (row < r0 || row >= r1) return;
  int L = __ldg(&p.context_lens[b]);
  L = L < 0 ? 0 : min(L, p.max_blocks * p.bs);
  const int pos = L - (r1 - r0) + (row - r0);
  const int h = hq / p.G;
  const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) + ((size_t)row * p.Hq + hq) * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(qrow[d]) * p.qscale;
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
      s = acc * __ldg(&p.k_scale[(size_t)blk * p.scale_row + h]);
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
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + ((size_t)row * p.Hq + hq) * D + lane * DPL;
#pragma unroll
  for (int d = 0; d < DPL; ++d) orow[d] = __float2bfloat16_rn(o[d] * inv);
}

}  // namespace

unsigned fetch_status_prefill_fp8_blocks() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_prefill_fp8, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v && cudaMemcpyToSymbol(g_status_prefill_fp8, &zero, sizeof(zero)) != cudaSuccess) return 0xffffffffu;
  return v;
}

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
      (long long)max_blocks_per_seq * block_size > 0x7fffffffll)
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
  const dim3 grid((unsigned)total_queries, (unsigned)groups);
  if (head_dim == 128)
    rows_kernel<128><<<grid, kRowWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else if (head_dim == 64)
    rows_kernel<64><<<grid, kRowWarps * 32, 0, (cudaStream_t)stream>>>(p);
  else
    rows_kernel<32><<<grid, kRowWarps * 32, 0, (cudaStream_t)stream>>>(p);
  return ck(cudaGetLastError(), "launch rows_kernel") ? PA_OK : PA_ERR_CUDA;
}
