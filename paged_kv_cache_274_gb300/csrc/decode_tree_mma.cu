// Drafted-tree decode kernel instances, mma.sync tiles of up to 16 query rows.
#include "paged_decode.cuh"

namespace pkv {

template <int D, int BS, bool FP8, bool I8>
static const void* tree_instance(int gt) {
  if (gt <= 8) return reinterpret_cast<const void*>(&paged_decode_kernel<D, BS, FP8, PKV_MATH_MMA, 8, I8, true, true>);
  if (gt <= 16) return reinterpret_cast<const void*>(&paged_decode_kernel<D, BS, FP8, PKV_MATH_MMA, 16, I8, true, true>);
  return nullptr;
}

// gt: query rows per tile
const void* decode_kernel_tree_mma(int kv_dtype, int D, int bs, int gt) {
  if (kv_dtype == PKV_KV_BF16) {
    if (D == 64) return bs == 16 ? tree_instance<64, 16, false, false>(gt) : tree_instance<64, 32, false, false>(gt);
    return bs == 16 ? tree_instance<128, 16, false, false>(gt) : tree_instance<128, 32, false, false>(gt);
  }
  if (kv_dtype == PKV_KV_FP8_E4M3)
    return bs == 16 ? tree_instance<128, 16, true, false>(gt) : tree_instance<128, 32, true, false>(gt);
  return bs == 16 ? tree_instance<128, 16, true, true>(gt) : tree_instance<128, 32, true, true>(gt);
}

}  // namespace pkv
