// pa_decode_fp8_blocks.cu — decode kernel instances for e4m3 K/V pools with one
// scale per (block, KV head).
//
// The kernel is the one in pa_decode_kernel.cuh with KT = fp8e4m3b: with each
// stage the producer moves the 16-byte chunk of the block's scale row that
// holds the item's heads, and a consumer warp reads its head's one value for
// all of the block's tokens.  Queries and output are bf16.  Compiled on its
// own so the instances build in parallel with the others.
#include "pa_decode_kernel.cuh"

namespace pa {
namespace {

using B16 = __nv_bfloat16;

// CUDA-core instances: 1 or 2 KV heads per item.
template <int D, int GT>
Launch pick_hg(int hg) {
  const void* merge = reinterpret_cast<const void*>(&merge_kernel<B16, D>);
  if (hg == 2) return {reinterpret_cast<const void*>(&decode_kernel<B16, fp8e4m3b, D, GT, false, 2>), merge};
  return {reinterpret_cast<const void*>(&decode_kernel<B16, fp8e4m3b, D, GT, false, 1>), merge};
}

template <int D>
Launch pick_gt(int gt, int hg) {
  if (gt == 4) return pick_hg<D, 4>(hg);
  if (gt == 2) return pick_hg<D, 2>(hg);
  return pick_hg<D, 1>(hg);
}

// Tensor-core instances (head_dim 128): GT query heads per KV head, 1 or 2 KV heads per item.
template <int GT>
Launch pick_mma_hg(int hg) {
  const void* merge = reinterpret_cast<const void*>(&merge_kernel<B16, 128>);
  if (hg == 2) return {reinterpret_cast<const void*>(&decode_kernel<B16, fp8e4m3b, 128, GT, true, 2>), merge};
  return {reinterpret_cast<const void*>(&decode_kernel<B16, fp8e4m3b, 128, GT, true, 1>), merge};
}

}  // namespace

Launch pick_decode_fp8_blocks(int head_dim, int gt, int hg, bool mma) {
  if (mma) {
    if (gt == 16) return pick_mma_hg<16>(hg);
    if (gt == 8) return pick_mma_hg<8>(hg);
    if (gt == 4) return pick_mma_hg<4>(hg);
    return pick_mma_hg<2>(hg);
  }
  if (head_dim == 32) return pick_gt<32>(gt, hg);
  if (head_dim == 64) return pick_gt<64>(gt, hg);
  return pick_gt<128>(gt, hg);
}

unsigned fetch_status_decode_fp8_blocks() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_decode, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v && cudaMemcpyToSymbol(g_status_decode, &zero, sizeof(zero)) != cudaSuccess) return 0xffffffffu;
  return v;
}

}  // namespace pa
