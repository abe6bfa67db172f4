// Visibility of drafted-tree nodes inside the attention kernels.
//
// A sequence of n cached tokens whose last m are the nodes of a drafted tree
// has base = n - m tokens before the tree.  A live row (query node t < m)
// attends to every position j < base, and to position base + u of the nodes u
// whose bit is set in row t of the tree mask (32 nodes per word).  The kernels
// work on windows of consecutive positions (a page, a step of 64 or 128
// tokens), so all they need is the 32 bits of a bit row from any bit on.
#pragma once

#include <cstdint>

namespace pkv {

// What the attention kernels know about the trees (all NULL / 0 outside
// pkv_paged_decode_tree).
struct TreeArgs {
  const uint32_t* mask;       // [B or 1][T][words] node visibility
  const int32_t* node_counts; // [B] nodes of each sequence; NULL: T each
  // [B][Hkv][words] nodes whose V row holds a NaN or an infinity (written by
  // the planner; NULL for INT8 caches, whose every code is finite)
  const uint32_t* poison;
  int words;                  // ceil(T / 32)
  int stride;                 // words between sequences of `mask` (0: one tree for all)
};

// Bits u0 .. u0 + 31 of a bit row of `words` words; bits before 0 and past the
// row are 0.
__device__ __forceinline__ uint32_t tree_window32(const uint32_t* row, int words, int u0) {
  const int w = u0 >> 5;  // floor, also for negative u0
  const uint32_t lo = (w >= 0 && w < words) ? __ldg(row + w) : 0u;
  const uint32_t hi = (w + 1 >= 0 && w + 1 < words) ? __ldg(row + w + 1) : 0u;
  return __funnelshift_r(lo, hi, u0 & 31);
}

__device__ __forceinline__ uint64_t tree_window64(const uint32_t* row, int words, int u0) {
  return static_cast<uint64_t>(tree_window32(row, words, u0)) |
         (static_cast<uint64_t>(tree_window32(row, words, u0 + 32)) << 32);
}

// The lowest n bits (n <= 0: none, n >= 64: all).
__device__ __forceinline__ uint64_t low_bits64(int n) {
  return n >= 64 ? ~0ull : (n <= 0 ? 0ull : ((1ull << n) - 1ull));
}
__device__ __forceinline__ uint32_t low_bits32(int n) {
  return n >= 32 ? ~0u : (n <= 0 ? 0u : ((1u << n) - 1u));
}

// What a row's output is besides O / l.  A row past the sequence's nodes is
// zero whatever its tile's products held (0 x NaN of a V row that other rows
// attend to is NaN); a row that attends to a node whose V row is not finite is
// NaN (those V rows are left out of the products, which would spread them to
// every row of the tile).
enum TreeRow : int { kTreeRowNormal = 0, kTreeRowZero = 1, kTreeRowNan = 2 };
__device__ __forceinline__ float tree_row_value(int state) { return state == kTreeRowNan ? __int_as_float(0x7fffffff) : 0.f; }

}  // namespace pkv
