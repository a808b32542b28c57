// pa_decode_fp8_blocks.cu — decode kernel instances for e4m3 K/V pools with one
// scale per (block, KV head).
//
// Blocks of 8 to 32 whose KV heads fill whole rows of 128 codes run
// tc_decode_kernel (pa_decode_tc.cuh), the rest direct_decode_kernel
// (pa_decode_direct.cuh).  Queries and output are bf16.  Compiled on its own so
// the instances build in parallel with the others.
#include "pa_decode_direct.cuh"
#include "pa_decode_tc.cuh"

namespace pa {
namespace {

using B16 = __nv_bfloat16;

template <int D>
Launch pick_direct(int gt) {
  const void* fin = reinterpret_cast<const void*>(&merge_wide_kernel<B16, D>);
  if (gt > 2) return {reinterpret_cast<const void*>(&direct_decode_kernel<B16, fp8e4m3b, D, 4, false>), fin};
  if (gt > 1) return {reinterpret_cast<const void*>(&direct_decode_kernel<B16, fp8e4m3b, D, 2, false>), fin};
  return {reinterpret_cast<const void*>(&direct_decode_kernel<B16, fp8e4m3b, D, 1, false>), fin};
}

// tcgen05 instances: gt query heads per CTA, 128 / head_dim KV heads per row of codes.
template <int GT, int HP>
Launch pick_tc(size_t* smem) {
  *smem = tc_smem_bytes<GT, HP>();
  return {reinterpret_cast<const void*>(&tc_decode_kernel<GT, HP, false>),
          reinterpret_cast<const void*>(&merge_wide_kernel<B16, 128 / HP>)};
}

template <int HP>
Launch pick_tc_gt(int gt, size_t* smem) {
  if (gt > 8) return pick_tc<16, HP>(smem);
  if (gt > 4) return pick_tc<8, HP>(smem);
  if constexpr (HP == 1)
    if (gt == 1) return pick_tc<1, HP>(smem);
  if constexpr (HP <= 2)
    if (gt <= 2) return pick_tc<2, HP>(smem);
  return pick_tc<4, HP>(smem);
}

}  // namespace

Launch pick_decode_fp8_blocks(int head_dim, int gt) {
  if (head_dim == 32) return pick_direct<32>(gt);
  if (head_dim == 64) return pick_direct<64>(gt);
  return pick_direct<128>(gt);
}

Launch pick_decode_fp8_blocks_tc(int head_dim, int gt, size_t* smem) {
  if (head_dim == 32) return pick_tc_gt<4>(gt, smem);
  if (head_dim == 64) return pick_tc_gt<2>(gt, smem);
  return pick_tc_gt<1>(gt, smem);
}

unsigned* status_word_decode_fp8_blocks() { return device_word(g_status_decode); }

}  // namespace pa
