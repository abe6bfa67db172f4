// Node masks and positions of drafted trees, from the nodes' parents.
//
// Node t of a tree sees itself and whatever its parent sees.  With m_0[t] =
// {t} and j_0[t] = parent[t], one round of pointer doubling
//   m_{r+1}[t] = m_r[t] | m_r[j_r[t]],   j_{r+1}[t] = j_r[j_r[t]]
// doubles the ancestors covered, so a tree of depth d takes ceil(log2(d + 1))
// rounds (9 for a chain of 512) instead of a walk of d dependent loads per
// node.  A node's depth is the number of bits of its row less one, and its
// position the tokens before the tree plus its depth.
//
// One CTA per sequence, a thread per (node, word of 32 nodes), both halves of
// the double buffer in shared memory.  The work is a few KB per tree: a call
// is one launch, and bound by its latency (3 us a call for one tree of 16
// nodes, where the host's part is as long; 4 to 7 us for 512 trees of 64).
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

__global__ void __launch_bounds__(1024) tree_masks_kernel(const TreeMaskArgs a) {
  extern __shared__ uint32_t sm[];
  pdl_trigger();
  pdl_wait();
  const int T = a.T, W = (T + 31) / 32, TW = T * W;
  uint32_t* mask[2] = {sm, sm + TW};
  int* jump[2] = {reinterpret_cast<int*>(sm + 2 * TW), reinterpret_cast<int*>(sm + 2 * TW) + T};
  const int b = blockIdx.x, tid = threadIdx.x;
  const int32_t* parents = a.parents + static_cast<size_t>(b) * T;
  // (all loads at once, also of nodes that are none: a thread per node at least)
  int nodes = a.node_counts != nullptr ? a.node_counts[b] : T;
  const int ctx = a.context_lens != nullptr ? a.context_lens[b] : nodes;
  int p = tid < T ? parents[tid] : -1;
  bool bad = nodes < 0 || nodes > T;
  if (bad) nodes = 0;
  for (int e = tid; e < TW; e += blockDim.x) {
    const int t = e / W, w = e - t * W;
    mask[0][e] = (t < nodes && (t >> 5) == w) ? 1u << (t & 31) : 0u;
  }
  bool more = false;
  if (tid < nodes) {
    if (p < -1 || p >= tid) {  // a parent comes before its children; else the node stands alone
      bad = true;
      p = -1;
    }
    jump[0][tid] = p;
    more = p >= 0;
  }
  int cur = 0;
  // at most 9 rounds: every jump of round r spans 2^r >= T nodes by then
  for (int r = 0; __syncthreads_or(more) && r < 10; ++r) {
    more = false;
    for (int e = tid; e < nodes * W; e += blockDim.x) {
      const int t = e / W, w = e - t * W;
      const int j = jump[cur][t];
      mask[cur ^ 1][e] = mask[cur][e] | (j >= 0 ? mask[cur][j * W + w] : 0u);
      if (w == 0) {
        const int jj = j >= 0 ? jump[cur][j] : -1;
        jump[cur ^ 1][t] = jj;
        more |= jj >= 0;
      }
    }
    cur ^= 1;
  }
  // (the loop's last barrier also ordered the last round's writes)
  uint32_t* out = a.mask + static_cast<size_t>(b) * TW;
  for (int e = tid; e < TW; e += blockDim.x) out[e] = e < nodes * W ? mask[cur][e] : 0u;
  if (a.positions != nullptr) {
    const int base = (a.context_lens != nullptr ? ctx : nodes) - nodes;
    for (int t = tid; t < T; t += blockDim.x) {
      int depth = -1;
      if (t < nodes)
        for (int w = 0; w < W; ++w) depth += __popc(mask[cur][t * W + w]);
      a.positions[static_cast<size_t>(b) * T + t] = t < nodes ? max(0, base + depth) : 0;
    }
  }
  if (bad) atomicOr(a.err, PKV_DEVERR_TREE);
}

cudaError_t launch_tree_masks(const TreeMaskArgs& a, cudaStream_t stream) {
  const int W = (a.T + 31) / 32;
  const size_t smem = sizeof(uint32_t) * 2 * (static_cast<size_t>(a.T) * W + a.T);  // 68 KB at T = 512
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(tree_masks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(static_cast<unsigned>(std::min(1024, (a.T * W + 31) / 32 * 32)));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_masks_kernel, a);
}

}  // namespace pkv
