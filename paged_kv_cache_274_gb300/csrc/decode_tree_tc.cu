// Drafted-tree decode kernel instances on tcgen05 (head_dim 128): one 128-row
// tile per CTA, and pairs of tiles (bf16 caches).
#include "paged_decode_tc.cuh"
#include "paged_decode_tc2.cuh"

namespace pkv {

template <int KV>
static const void* tree_tc_instance(int bs, bool rot) {
  if (bs == 16) return rot ? reinterpret_cast<const void*>(&paged_decode_tc_kernel<16, true, KV, true>)
                           : reinterpret_cast<const void*>(&paged_decode_tc_kernel<16, false, KV, true>);
  return rot ? reinterpret_cast<const void*>(&paged_decode_tc_kernel<32, true, KV, true>)
             : reinterpret_cast<const void*>(&paged_decode_tc_kernel<32, false, KV, true>);
}

// rot: tiles of at most 96 query rows, rotated into the highest TMEM lanes
const void* decode_kernel_tree_tc(int bs, bool rot, int kv_dtype) {
  if (kv_dtype == PKV_KV_FP8_E4M3) return tree_tc_instance<PKV_KV_FP8_E4M3>(bs, rot);
  if (kv_dtype == PKV_KV_INT8) return tree_tc_instance<PKV_KV_INT8>(bs, rot);
  return tree_tc_instance<PKV_KV_BF16>(bs, rot);
}

const void* decode_kernel_tree_tc2(int bs) {
  return bs == 16 ? reinterpret_cast<const void*>(&paged_decode_tc2_kernel<16, true>)
                  : reinterpret_cast<const void*>(&paged_decode_tc2_kernel<32, true>);
}

}  // namespace pkv
