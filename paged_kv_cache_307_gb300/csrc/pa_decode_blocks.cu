// pa_decode_blocks.cu — host side of decode over block-scaled e4m3 pools
// (pa_decode_fp8_blocks) and of the decode that keeps the softmax weights
// (pa_decode_weights).
//
// Which kernel: block-scaled pools whose KV heads fill whole rows of 128 codes, in
// blocks of 8 and more, run tc_decode_kernel (pa_decode_tc.cuh); bf16 query groups
// keep pa_decode's tensor-core kernel in weights mode (decode_weights_mma); the
// rest runs direct_decode_kernel (pa_decode_direct.cuh).  Partitions are merged,
// and weights added, by merge_wide_kernel or weights_kernel (pa_decode_kernel.cuh).
#include "pa_decode_kernel.cuh"

namespace pa {
namespace {

enum class Form { kTc, kMma, kDirect };

bool tc_shape(int num_kv_heads, int head_dim, int block_size) {
  return block_size >= 8 && num_kv_heads % (128 / head_dim) == 0;    // (a TMA box is whole 8-row swizzle atoms)
}
// CTAs of the tcgen05 kernel that share a row of 128 codes, 16 query heads at most each.
int tc_subs(int G, int head_dim) { return (G * (128 / head_dim) + 15) / 16; }

Form form_of(pa_dtype kv, int G, int num_kv_heads, int head_dim, int block_size) {
  if (kv == PA_FP8_E4M3) return tc_shape(num_kv_heads, head_dim, block_size) ? Form::kTc : Form::kDirect;
  return kv == PA_BF16 && bf16_mma_shape(G, head_dim, block_size) ? Form::kMma : Form::kDirect;
}

bool good_sizes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_blocks, int block_size,
                int partition_size) {
  return num_seqs >= 0 && num_heads > 0 && num_kv_heads > 0 && num_heads % num_kv_heads == 0 &&
         supported_head_dim(head_dim) && supported_block_size(block_size) && max_blocks > 0 &&
         (long long)max_blocks * block_size <= kMaxRowTokens &&
         !(partition_size > 0 && partition_size % block_size) && (long long)num_seqs * num_heads <= 0x7fffffffll;
}

// Automatic split: the longest partition that still gives the GPU its CTAs at the
// table's capacity (the lengths themselves are on the device).
//  * tcgen05, one CTA per (partition, sequence, row of 128 codes): 2048, 1024 or 512
//    tokens, two CTAs per SM.  A CTA's start and end weigh about as much as two of
//    its 128-token tiles: 64 requests x 8 KV heads over U[1024, 16384] take 258, 204
//    and 188 us at 512, 1024 and 2048 tokens; one request x 8 heads at 32768 tokens
//    24.0, 20.7 and 29.2, eight at up to 8192 28.7, 23.8 and 28.6.
//  * direct, one CTA per (partition, sequence, KV head, 4 query heads): 512 down to
//    64 tokens, four CTAs per SM: 5 requests x 4 heads of up to 700 tokens (f32)
//    take 12.5, 14.6, 22.8 and 39.2 us at 64, 128, 256 and 512 tokens; 32 x 8 heads
//    over U[128, 4096] (bf16, groups of 3) 120, 103, 96 and 91.
//  * mma: pa_decode's own.
int partition_of(Form form, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_blocks, int bs,
                 int partition_size) {
  if (form == Form::kMma)
    return pa_decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, bs, partition_size);
  const int max_ctx = max_blocks * bs;
  if (partition_size < 0) return max_ctx;
  int P = partition_size;
  if (P <= 0) {
    const int G = num_heads / num_kv_heads;
    const bool tc = form == Form::kTc;
    const long long items = tc ? (long long)num_seqs * (num_kv_heads / (128 / head_dim)) * tc_subs(G, head_dim)
                               : (long long)num_seqs * num_kv_heads * ((G + 3) / 4);
    const int least = tc ? 512 : 64;
    P = tc ? 2048 : 512;
    while (P > least && items * max_ctx < (tc ? 2ll : 4ll) * kTunedSms * P) P /= 2;
  }
  return P >= max_ctx ? max_ctx : P;
}

int run(void* out, const void* query, const void* k_cache, const void* v_cache, const float* k_scale,
        const float* v_scale, const int32_t* block_tables, int max_blocks, const int32_t* context_lens, int num_seqs,
        int num_heads, int num_kv_heads, int head_dim, int bs, int num_blocks, float scale, int partition_size,
        void* workspace, size_t workspace_bytes, pa_dtype dtype, pa_dtype kv, float* weights, long long stride,
        bool keep, void* stream) {
  if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
  const bool fp8 = kv == PA_FP8_E4M3;
  if (fp8 ? dtype != PA_BF16 : kv != dtype) return PA_ERR_DTYPE;
  if (!good_sizes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, bs, partition_size) || num_blocks <= 0)
    return PA_ERR_SHAPE;
  const long long max_ctx = (long long)max_blocks * bs;
  const int G = num_heads / num_kv_heads;
  const Form form = form_of(kv, G, num_kv_heads, head_dim, bs);
  const int P = partition_of(form, num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, bs, partition_size);
  const int max_parts = (int)((max_ctx + P - 1) / P);
  const int hp = 128 / head_dim;
  const int nsub = form == Form::kTc ? tc_subs(G, head_dim) : (G + 3) / 4;
  const long long ctas = (long long)max_parts * num_seqs * nsub * (form == Form::kTc ? num_kv_heads / hp : num_kv_heads);
  const long long second = (long long)num_seqs * num_heads +
                           (long long)num_seqs * num_kv_heads * ((max_ctx + kWeightTokens - 1) / kWeightTokens);
  if (ctas > 0x7fffffffll || (keep && (stride < max_ctx || G > 1024 || second > 0x7fffffffll))) return PA_ERR_SHAPE;
  if (num_seqs == 0) return PA_OK;
  if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens || (keep && !weights) ||
      (fp8 && (!k_scale || !v_scale)))
    return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (fp8 && (!aligned16(k_scale) || !aligned16(v_scale))))
    return PA_ERR_ALIGN;
  const long long rows = (long long)num_seqs * num_heads;
  const size_t partials = keep || max_parts > 1 ? partials_bytes(rows, max_parts, head_dim) : 0;
  const size_t need = partials + (keep ? (size_t)(rows * max_ctx * 4) : 0);
  if (need && !aligned16(workspace)) return PA_ERR_ALIGN;
  if (need && (!workspace || workspace_bytes < need)) return PA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const WeightsArgs wa{weights, stride, keep ? reinterpret_cast<float*>(ws + partials) : nullptr};
  if (form == Form::kMma)
    return decode_weights_mma(out, query, k_cache, v_cache, block_tables, max_blocks, context_lens, num_seqs,
                              num_heads, num_kv_heads, head_dim, bs, num_blocks, scale, partition_size, workspace,
                              partials, wa, stream);

  DecodeParams prm = {};
  prm.out = out;
  prm.q = query;
  prm.block_tables = block_tables;
  prm.context_lens = context_lens;
  prm.ws_ml = need ? reinterpret_cast<float*>(ws) : nullptr;
  prm.ws_o = need ? reinterpret_cast<float*>(ws + (rows * max_parts * 8 + 255) / 256 * 256) : nullptr;
  prm.ws_s = wa.scores;
  prm.B = num_seqs;
  prm.Hq = num_heads;
  prm.Hkv = num_kv_heads;
  prm.G = G;
  prm.nsub = nsub;
  prm.max_blocks = max_blocks;
  prm.bs = bs;
  prm.num_blocks = num_blocks;
  prm.part_tokens = P;
  prm.max_parts = max_parts;
  prm.qscale = scale * kLog2e;
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.scale_row = scale_row(num_kv_heads);
  prm.k_codes = static_cast<const uint8_t*>(k_cache);
  Launch L;
  if (form == Form::kTc) {
    int dev = 0;
    if (!ck(cudaGetDevice(&dev), "cudaGetDevice")) return PA_ERR_CUDA;
    CUtensorMap mapK, mapV;
    if (!pool_map(&mapK, k_cache, kv, num_blocks, bs, num_kv_heads / hp, 128, dev, true, 1) ||
        !pool_map(&mapV, v_cache, kv, num_blocks, bs, num_kv_heads / hp, 128, dev, true, 1)) {
      note_host_error("cuTensorMapEncodeTiled failed for the K/V pool");
      return PA_ERR_CUDA;
    }
    const int gt = (hp * G + nsub - 1) / nsub;
    size_t smem = 0;
    L = keep ? pick_decode_weights_fp8_tc(head_dim, gt, &smem) : pick_decode_fp8_blocks_tc(head_dim, gt, &smem);
    if (!raise_smem_limit(L.kernel, dev)) return PA_ERR_CUDA;
    void* args[] = {&mapK, &mapV, &prm};
    if (!ck(cudaLaunchKernel(L.kernel, dim3((unsigned)ctas), dim3(kTcThreads), args, smem, (cudaStream_t)stream),
            "cudaLaunchKernel(tc_decode_kernel)"))
      return PA_ERR_CUDA;
  } else {
    const int gt = (G + nsub - 1) / nsub;
    L = !keep ? pick_decode_fp8_blocks(head_dim, gt)
        : fp8 ? pick_decode_weights_fp8(head_dim, gt)
              : pick_decode_weights(dtype == PA_F32, head_dim, gt);
    void* args[] = {&prm, &k_cache, &v_cache};
    if (!ck(cudaLaunchKernel(L.kernel, dim3((unsigned)ctas), dim3(kDirectThreads), args, 0, (cudaStream_t)stream),
            "cudaLaunchKernel(direct_decode_kernel)"))
      return PA_ERR_CUDA;
  }
  if (keep) return launch_weights(L, prm, wa, stream);
  if (max_parts > 1) {
    void* args[] = {&prm};
    if (!ck(launch_dependent(L.merge, dim3(merge_ctas_of(prm)), dim3(kFinishThreads), args, 0, (cudaStream_t)stream),
            "cudaLaunchKernel(merge_wide_kernel)"))
      return PA_ERR_CUDA;
  }
  return PA_OK;
}

// 0 for sizes that the calls refuse.
size_t bytes_of(pa_dtype kv, bool keep, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_blocks,
                int bs, int partition_size) {
  if (!good_sizes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, bs, partition_size) || num_seqs == 0)
    return 0;
  const Form form = form_of(kv, num_heads / num_kv_heads, num_kv_heads, head_dim, bs);
  const int P = partition_of(form, num_seqs, num_heads, num_kv_heads, head_dim, max_blocks, bs, partition_size);
  const long long max_ctx = (long long)max_blocks * bs, rows = (long long)num_seqs * num_heads;
  const int max_parts = (int)((max_ctx + P - 1) / P);
  return (keep || max_parts > 1 ? partials_bytes(rows, max_parts, head_dim) : 0) +
         (keep ? (size_t)(rows * max_ctx * 4) : 0);
}

}  // namespace

int launch_weights(const Launch& L, const DecodeParams& prm, const WeightsArgs& wa, void* stream) {
  DecodeParams p = prm;
  float* w = wa.weights;
  long long stride = wa.stride;
  unsigned merge_ctas = merge_ctas_of(p);
  const long long max_ctx = (long long)p.max_blocks * p.bs;
  // one wave of CTAs at the table's capacity (eight fit an SM) where the chunks allow it
  const long long all = (long long)p.B * p.Hkv * ((max_ctx + kWeightTokens - 1) / kWeightTokens);
  int chunks = (int)(all / (8 * device_sm_count()));
  chunks = chunks < 1 ? 1 : chunks > 8 ? 8 : chunks;
  const long long span = (long long)chunks * kWeightTokens;
  const long long ctas = merge_ctas + (long long)p.B * p.Hkv * ((max_ctx + span - 1) / span);
  void* args[] = {&p, &w, &stride, &merge_ctas, &chunks};
  return ck(launch_dependent(L.merge, dim3((unsigned)ctas), dim3(kFinishThreads), args, 2 * (size_t)p.G * 4,
                             (cudaStream_t)stream),
            "cudaLaunchKernel(weights_kernel)")
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace pa

using namespace pa;

extern "C" int pa_decode_fp8_blocks(void* out, const void* query, const void* k_cache, const void* v_cache,
                                    const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                                    int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                    float scale, int partition_size, void* workspace, size_t workspace_bytes,
                                    pa_dtype dtype, void* stream) {
  return run(out, query, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks_per_seq, context_lens, num_seqs,
             num_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, partition_size, workspace,
             workspace_bytes, dtype, PA_FP8_E4M3, nullptr, 0, false, stream);
}

extern "C" int pa_decode_weights(void* out, float* weights, long long weights_stride, const void* query,
                                 const void* k_cache, const void* v_cache, const float* k_scale,
                                 const float* v_scale, const int32_t* block_tables, int max_blocks_per_seq,
                                 const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                                 int head_dim, int block_size, int num_blocks, float scale, int partition_size,
                                 void* workspace, size_t workspace_bytes, pa_dtype dtype, pa_dtype kv_dtype,
                                 void* stream) {
  return run(out, query, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks_per_seq, context_lens, num_seqs,
             num_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, partition_size, workspace,
             workspace_bytes, dtype, kv_dtype, weights, weights_stride, true, stream);
}

extern "C" int pa_decode_fp8_blocks_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                   int max_blocks_per_seq, int block_size, int partition_size) {
  if (!good_sizes(num_seqs, num_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size, partition_size))
    return PA_ERR_SHAPE;
  return partition_of(form_of(PA_FP8_E4M3, num_heads / num_kv_heads, num_kv_heads, head_dim, block_size), num_seqs,
                      num_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size, partition_size);
}

extern "C" size_t pa_decode_fp8_blocks_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                       int max_blocks_per_seq, int block_size, int partition_size) {
  return bytes_of(PA_FP8_E4M3, false, num_seqs, num_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                  partition_size);
}

extern "C" size_t pa_decode_weights_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                    int max_blocks_per_seq, int block_size, int partition_size,
                                                    pa_dtype kv_dtype) {
  return bytes_of(kv_dtype, true, num_seqs, num_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                  partition_size);
}
