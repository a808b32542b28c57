// pa_latent_decode.cu — attention over a paged cache of one latent vector a token, in the
// absorbed form (pa_latent_decode): the rows are the keys, and their latent part the values.
//
// One CTA per (query row, head): scores of 64 tokens at a time by the warps, a running maximum
// and sum, and a thread per two latent elements for the values.
#include "pa_common.cuh"

namespace pa {
namespace {

__device__ unsigned g_status_latent;

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct LatentParams {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const __nv_bfloat16* cache;
  const int32_t* query_start;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int B, H, R, P, rows, max_blocks, bs, num_blocks;
  float qscale;
};

__global__ void __launch_bounds__(kThreads) latent_decode_kernel(const LatentParams p) {
  __shared__ float qs[576], sc[kTile];
  __shared__ const __nv_bfloat16* at[kTile];
  const int row = blockIdx.x / p.H, h = blockIdx.x % p.H;
  int b = row, i = 0, n = 1;
  if (p.query_start) {
    int a = 0, e = 0;
    bool found = false, bad = false;
    for (int s = 0; s < p.B; ++s) {
      const int x = p.query_start[s], y = p.query_start[s + 1];
      const bool ok = x >= 0 && y >= x && y <= p.rows;
      bad |= !ok;
      if (ok && row >= x && row < y) {
        b = s;
        a = x;
        e = y;
        found = true;
      }
    }
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status_latent, PA_DEV_BAD_LEN);
    if (!found) return;
    i = row - a;
    n = e - a;
    if (i < 0 || i >= n) return;
  }
  const int Lmax = p.max_blocks * p.bs;
  int L = p.context_lens[b];
  if (L < 0 || L > Lmax) {
    if (threadIdx.x == 0) atomicOr(&g_status_latent, PA_DEV_BAD_LEN);
    L = L < 0 ? 0 : Lmax;
  }
  const int end = L - n + i + 1;               // tokens that the row sees
  const int W = p.R + p.P;
  const size_t r = (size_t)row * p.H + h;
  for (int d = threadIdx.x; d < W; d += kThreads) qs[d] = __bfloat162float(p.q[r * W + d]);
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t0 = 0; t0 < end; t0 += kTile) {
    __syncthreads();
    const int nt = min(kTile, end - t0);
    for (int t = warp; t < nt; t += kThreads / 32) {
      int id = p.block_tables[(size_t)b * p.max_blocks + (t0 + t) / p.bs];
      if ((unsigned)id >= (unsigned)p.num_blocks) {
        if (lane == 0) atomicOr(&g_status_latent, PA_DEV_BAD_BLOCK);
        id = 0;
      }
      const __nv_bfloat16* c = p.cache + ((size_t)id * p.bs + (t0 + t) % p.bs) * W;
      float s = 0.f;
      for (int d = lane; d < W; d += 32) s = fmaf(qs[d], __bfloat162float(c[d]), s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (lane == 0) {
        sc[t] = s * p.qscale;
        at[t] = c;
      }
    }
    __syncthreads();
    float mx = m;
    for (int t = 0; t < nt; ++t) mx = fmaxf(mx, sc[t]);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mx);
    l *= f;
    o[0] *= f;
    o[1] *= f;
    m = mx;
    for (int t = 0; t < nt; ++t) {
      const float w = mx == -INFINITY ? 0.f : exp2f(sc[t] - mx);
      l += w;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (threadIdx.x + k * kThreads < p.R) o[k] = fmaf(w, __bfloat162float(at[t][threadIdx.x + k * kThreads]), o[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (threadIdx.x + k * kThreads < p.R)
      p.out[r * p.R + threadIdx.x + k * kThreads] = __float2bfloat16_rn(l != 0.f ? o[k] / l : 0.f);
}

bool good_sizes(int total, int num_seqs, int num_heads, int latent_dim, int max_blocks, int bs, int partition_size) {
  return total >= 0 && num_seqs >= 0 && num_heads > 0 && latent_shape(latent_dim, 16, bs) && max_blocks > 0 &&
         (long long)max_blocks * bs <= kMaxRowTokens && !(partition_size > 0 && partition_size % bs) &&
         (long long)total * num_heads <= 0x7fffffffll;
}

}  // namespace

unsigned* status_word_latent_decode() { return device_word(g_status_latent); }

}  // namespace pa

using namespace pa;

extern "C" int pa_latent_decode(void* out, const void* query, const int32_t* query_start, int total_queries,
                                const void* cache, const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* context_lens, int num_seqs, int num_heads, int latent_dim,
                                int rope_dim, int block_size, int num_blocks, float scale, int partition_size,
                                void* workspace, size_t workspace_bytes, pa_dtype dtype, void* stream) {
  if (dtype != PA_BF16) return PA_ERR_DTYPE;
  if (!good_sizes(total_queries, num_seqs, num_heads, latent_dim, max_blocks_per_seq, block_size, partition_size) ||
      !latent_shape(latent_dim, rope_dim, block_size) || num_blocks <= 0 || !(scale > 0.f) ||
      (!query_start && total_queries != num_seqs))
    return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_queries == 0) return PA_OK;
  if (!out || !query || !cache || !block_tables || !context_lens) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(cache)) return PA_ERR_ALIGN;
  LatentParams p = {};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q = static_cast<const __nv_bfloat16*>(query);
  p.cache = static_cast<const __nv_bfloat16*>(cache);
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.B = num_seqs;
  p.H = num_heads;
  p.R = latent_dim;
  p.P = rope_dim;
  p.rows = total_queries;
  p.max_blocks = max_blocks_per_seq;
  p.bs = block_size;
  p.num_blocks = num_blocks;
  p.qscale = scale * kLog2e;
  void* args[] = {&p};
  return ck(cudaLaunchKernel(reinterpret_cast<const void*>(&latent_decode_kernel),
                             dim3((unsigned)total_queries * num_heads), dim3(kThreads), args, 0, (cudaStream_t)stream),
            "cudaLaunchKernel(latent_decode_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}

extern "C" size_t pa_latent_decode_workspace_bytes(int total_queries, int num_seqs, int num_heads, int latent_dim,
                                                   int max_blocks_per_seq, int block_size, int partition_size) {
  return 0;
}

extern "C" int pa_latent_decode_partition_size(int total_queries, int num_seqs, int num_heads, int latent_dim,
                                               int max_blocks_per_seq, int block_size, int partition_size) {
  if (!good_sizes(total_queries, num_seqs, num_heads, latent_dim, max_blocks_per_seq, block_size, partition_size))
    return PA_ERR_SHAPE;
  return max_blocks_per_seq * block_size;
}
