// Work shares of the tcgen05 drafted-tree attention (written by its planner,
// read by the attention and the merge kernels).
#pragma once

#include <cstdint>

#include "pkv_internal.h"

namespace pkv {

constexpr int kTreeTokens = 128;  // tokens of a step

// Start of a share of the steps of all (sequence, KV head) items in a row.
struct TreeBound {
  int b, kvh;  // item (b = batch, kvh = 0: the end)
  int step;    // step of the item (0: the share starts with the item)
  int ctx;   // the sequence's validated length
};

}  // namespace pkv
