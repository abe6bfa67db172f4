// Drafted-tree nodes whose V row is not finite, found by extra CTAs of the
// planners.
//
// Such a row would reach every query row of a tile through 0 x NaN, also those
// that do not attend to the node, so the attention kernels leave these V rows
// out of the products and set the rows that attend to them to NaN.
//
// One warp per (sequence, KV head, word of 32 nodes): lane i finds node i's
// page, then a row takes row_bytes / 16 lanes, so the warp reads 2 or 4 rows at
// a time and all of a lane's loads (8 or 16) are in flight together.  The rows
// come out of L2 again when the attention reads the pages: T x Hkv rows a
// sequence, 4 MB for 64 sequences of 32 nodes and 8 KV heads of 256 bytes.
#pragma once

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

struct TreeScan {
  const int32_t* context_lens;
  const int32_t* node_counts;  // NULL: T each
  const int32_t* block_tables;
  const uint8_t* v;            // the cache slot's V pages
  uint32_t* poison;            // [B][Hkv][words]
  int B, T, words, Hkv, MB, NB, bs, row_bytes, e4m3;
};

// 16 bytes of a V row with a value that is not finite.  E4M3: NaN has every
// bit but the sign set; adding 1 to seven set bits carries into the eighth.
// bf16: the exponent is all ones; likewise with its lowest bit.
__device__ __forceinline__ bool not_finite(const uint4& x, bool e4m3) {
  const uint32_t bits = e4m3 ? 0x7f7f7f7fu : 0x7f807f80u, one = e4m3 ? 0x01010101u : 0x00800080u;
  const uint32_t top = e4m3 ? 0x80808080u : 0x80008000u;
  return ((((x.x & bits) + one) | ((x.y & bits) + one) | ((x.z & bits) + one) | ((x.w & bits) + one)) & top) != 0u;
}

template <int kLanes>  // lanes of one row
__device__ __forceinline__ uint32_t tree_scan_word(const TreeScan& t, int b, int h, int w, int n, int nodes) {
  constexpr int kRows = 32 / kLanes;  // rows at a time
  const int lane = threadIdx.x & 31, sub = lane / kLanes, chunk = lane % kLanes;
  // lane i: the first byte of node 32 w + i's row, -1 if there is none
  long long row = -1;
  {
    const int u = 32 * w + lane, pos = n - nodes + u;
    if (u < nodes && pos >= 0) {
      const int blk = t.block_tables[static_cast<size_t>(b) * t.MB + pos / t.bs];
      if (static_cast<unsigned>(blk) < static_cast<unsigned>(t.NB))
        row = ((static_cast<long long>(blk) * t.Hkv + h) * t.bs + pos % t.bs) * t.row_bytes;
    }
  }
  uint32_t word = 0u;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 8 * kRows) {
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long long at = __shfl_sync(kFull, row, (r0 + k * kRows + sub) & 31);
      x[k] = at >= 0 ? __ldcg(reinterpret_cast<const uint4*>(t.v + at + 16 * chunk)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t votes = __ballot_sync(kFull, not_finite(x[k], t.e4m3 != 0));
#pragma unroll
      for (int s = 0; s < kRows; ++s) {
        constexpr uint32_t kGroup = (1u << kLanes) - 1u;
        if ((votes >> (s * kLanes)) & kGroup) word |= 1u << ((r0 + k * kRows + s) & 31);
      }
    }
  }
  return word;
}

// Words warp0, warp0 + nwarps, ... of the B x Hkv x words.
__device__ __forceinline__ void tree_scan_values(const TreeScan& t, int warp0, int nwarps) {
  const unsigned items = static_cast<unsigned>(t.B) * t.Hkv * t.words;  // (less than 2^31, as the host checks)
#pragma unroll 1
  for (unsigned i = warp0; i < items; i += nwarps) {
    const int it = static_cast<int>(i), bh = it / t.words, w = it - bh * t.words;
    const int b = bh / t.Hkv, h = bh - b * t.Hkv;
    const int n = t.context_lens[b];
    const int nodes = t.node_counts != nullptr ? t.node_counts[b] : t.T;
    uint32_t word = 0u;
    if (n >= 0 && n <= t.MB * t.bs && nodes >= 0 && nodes <= t.T)
      word = t.row_bytes == 256 ? tree_scan_word<16>(t, b, h, w, n, nodes) : tree_scan_word<8>(t, b, h, w, n, nodes);
    if ((threadIdx.x & 31) == 0) t.poison[it] = word;
  }
}

inline TreeScan tree_scan_of(const DecodeLaunch& L, uint32_t* poison) {
  return TreeScan{L.context_lens, L.node_counts, L.block_tables, static_cast<const uint8_t*>(L.v_cache), poison,
                  L.B, L.T, L.tree_words, L.Hkv, L.MB, L.NB, L.bs, L.D * (L.kv_fp8 ? 1 : 2),
                  L.kv_dtype == PKV_KV_FP8_E4M3 ? 1 : 0};
}

// Planner CTAs for the scan (none for INT8 caches, whose every code is finite):
// a warp per word up to a full GPU.
inline unsigned tree_scan_ctas(const DecodeLaunch& L, int warps_per_cta) {
  if (L.kv_dtype == PKV_KV_INT8) return 0;
  const long long items = static_cast<long long>(L.B) * L.Hkv * L.tree_words;
  return static_cast<unsigned>(std::min<long long>((items + warps_per_cta - 1) / warps_per_cta, 151 * 32 / warps_per_cta));
}

}  // namespace pkv
