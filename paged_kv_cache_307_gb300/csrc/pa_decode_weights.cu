// pa_decode_weights.cu — weights-mode decode instances (scores kept for
// weights_kernel) for f32 and bf16 K/V pools.  Compiled on its own so the
// instances build in parallel with the others.
#include "pa_decode_direct.cuh"

namespace pa {
namespace {

using B16 = __nv_bfloat16;

template <typename T, int D>
Launch pick_direct(int gt) {
  const void* fin = reinterpret_cast<const void*>(&weights_kernel<T, D>);
  if (gt > 2) return {reinterpret_cast<const void*>(&direct_decode_kernel<T, T, D, 4, true>), fin};
  if (gt > 1) return {reinterpret_cast<const void*>(&direct_decode_kernel<T, T, D, 2, true>), fin};
  return {reinterpret_cast<const void*>(&direct_decode_kernel<T, T, D, 1, true>), fin};
}

template <typename T>
Launch pick_d(int d, int gt) {
  if (d == 32) return pick_direct<T, 32>(gt);
  if (d == 64) return pick_direct<T, 64>(gt);
  return pick_direct<T, 128>(gt);
}

// Tensor-core instances: bf16, head_dim 64 or 128, GT query heads per KV head.
template <int D, int GT>
Launch pick_mma_hg(int hg) {
  const void* fin = reinterpret_cast<const void*>(&weights_kernel<B16, D>);
  if (hg == 4) return {reinterpret_cast<const void*>(&decode_kernel<B16, B16, D, GT, true, 4, true>), fin};
  if (hg == 2) return {reinterpret_cast<const void*>(&decode_kernel<B16, B16, D, GT, true, 2, true>), fin};
  return {reinterpret_cast<const void*>(&decode_kernel<B16, B16, D, GT, true, 1, true>), fin};
}

template <int D>
Launch pick_mma(int gt, int hg) {
  if (gt == 16) return pick_mma_hg<D, 16>(hg);
  if (gt == 8) return pick_mma_hg<D, 8>(hg);
  if (gt == 4) return pick_mma_hg<D, 4>(hg);
  return pick_mma_hg<D, 2>(hg);
}

}  // namespace

Launch pick_decode_weights_mma(int head_dim, int gt, int hg) {
  return head_dim == 64 ? pick_mma<64>(gt, hg) : pick_mma<128>(gt, hg);
}

Launch pick_decode_weights(bool f32, int head_dim, int gt) {
  return f32 ? pick_d<float>(head_dim, gt) : pick_d<B16>(head_dim, gt);
}

unsigned* status_word_decode_weights() { return device_word(g_status_decode); }

}  // namespace pa
