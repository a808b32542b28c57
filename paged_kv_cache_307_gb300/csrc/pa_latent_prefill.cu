// pa_latent_prefill.cu — ragged causal attention over expanded latent vectors
// (pa_latent_prefill): keys of key_dim elements a head and one rotated key for all heads.
//
// One CTA per (query row, head): scores of 64 tokens at a time by the warps, a running maximum
// and sum, and a thread per element for the values.
#include "pa_common.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_latent;

constexpr int kThreads = 128;
constexpr int kTile = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct LatentParams {
  __nv_bfloat16* out;
  const __nv_bfloat16 *q, *kv, *key;
  const int32_t *query_start, *kv_start;
  long long key_stride;
  int B, H, Dk, P, Dv, rows, kv_rows;
  float qscale;
};

__global__ void __launch_bounds__(kThreads) latent_prefill_kernel(const LatentParams p) {
  __shared__ float qs[192], sc[kTile];
  const int row = blockIdx.x / p.H, h = blockIdx.x % p.H;
  int a = 0, e = 0, k0 = 0, k1 = 0;
  bool found = false, bad = false;
  for (int s = 0; s < p.B; ++s) {
    const int x = p.query_start[s], y = p.query_start[s + 1], u = p.kv_start[s], v = p.kv_start[s + 1];
    const bool ok = x >= 0 && y >= x && y <= p.rows && u >= 0 && v >= u && v <= p.kv_rows;
    bad |= !ok;
    if (ok && row >= x && row < y) {
      a = x;
      e = y;
      k0 = u;
      k1 = v;
      found = true;
    }
  }
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status_latent, PA_DEV_BAD_LEN);
  if (!found) return;
  const int end = (k1 - k0) - (e - a) + (row - a) + 1;
  const int W = p.Dk + p.P, KV = p.Dk + p.Dv;
  const size_t r = (size_t)row * p.H + h;
  for (int d = threadIdx.x; d < W; d += kThreads) qs[d] = __bfloat162float(p.q[r * W + d]);
  float m = -INFINITY, l = 0.f, o = 0.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t0 = 0; t0 < end; t0 += kTile) {
    __syncthreads();
    const int nt = min(kTile, end - t0);
    for (int t = warp; t < nt; t += kThreads / 32) {
      const __nv_bfloat16* k = p.kv + ((size_t)(k0 + t0 + t) * p.H + h) * KV;
      const __nv_bfloat16* kr = p.key + (k0 + t0 + t) * p.key_stride;
      float s = 0.f;
      for (int d = lane; d < W; d += 32) s = fmaf(qs[d], __bfloat162float(d < p.Dk ? k[d] : kr[d - p.Dk]), s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (lane == 0) sc[t] = s * p.qscale;
    }
    __syncthreads();
    float mx = m;
    for (int t = 0; t < nt; ++t) mx = fmaxf(mx, sc[t]);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mx);
    l *= f;
    o *= f;
    m = mx;
    for (int t = 0; t < nt; ++t) {
      const float w = mx == -INFINITY ? 0.f : exp2f(sc[t] - mx);
      l += w;
      if (threadIdx.x < p.Dv)
        o = fmaf(w, __bfloat162float(p.kv[((size_t)(k0 + t0 + t) * p.H + h) * KV + p.Dk + threadIdx.x]), o);
    }
  }
  if (threadIdx.x < p.Dv) p.out[r * p.Dv + threadIdx.x] = __float2bfloat16_rn(l != 0.f ? o / l : 0.f);
}

bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

}  // namespace

unsigned* status_word_latent_prefill() { return device_word(g_status_latent); }

}  // namespace pa

using namespace pa;

extern "C" int pa_latent_prefill(void* out, const void* query, const int32_t* query_start, int total_queries,
                                 const void* kv, const void* key_rope, long long key_rope_stride,
                                 const int32_t* kv_start, int total_kv, int num_seqs, int num_heads, int key_dim,
                                 int rope_dim, int value_dim, float scale, pa_dtype dtype, void* stream) {
  if (dtype != PA_BF16) return PA_ERR_DTYPE;
  if (total_queries < 0 || total_kv < 0 || num_seqs < 0 || num_seqs > 2048 || num_heads <= 0 || !dim_ok(key_dim) ||
      !dim_ok(value_dim) || rope_dim <= 0 || rope_dim > 64 || rope_dim % 16 || key_rope_stride < rope_dim ||
      !(scale > 0.f) || (long long)total_queries * num_heads > 0x7fffffffll)
    return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_queries == 0) return PA_OK;
  if (!out || !query || !query_start || !kv_start || (total_kv && (!kv || !key_rope))) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(kv) || !aligned16(key_rope) || key_rope_stride % 8)
    return PA_ERR_ALIGN;
  LatentParams p = {};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q = static_cast<const __nv_bfloat16*>(query);
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.key = static_cast<const __nv_bfloat16*>(key_rope);
  p.query_start = query_start;
  p.kv_start = kv_start;
  p.key_stride = key_rope_stride;
  p.B = num_seqs;
  p.H = num_heads;
  p.Dk = key_dim;
  p.P = rope_dim;
  p.Dv = value_dim;
  p.rows = total_queries;
  p.kv_rows = total_kv;
  p.qscale = scale * kLog2e;
  void* args[] = {&p};
  return ck(cudaLaunchKernel(reinterpret_cast<const void*>(&latent_prefill_kernel),
                             dim3((unsigned)total_queries * num_heads), dim3(kThreads), args, 0, (cudaStream_t)stream),
            "cudaLaunchKernel(latent_prefill_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}
