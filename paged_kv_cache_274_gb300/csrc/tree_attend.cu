// Planner and launch of the tcgen05 drafted-tree attention
// (tree_attend.cuh), and its kernel instances.
#include <algorithm>
#include <mutex>
#include <type_traits>
#include <vector>

#include "tree_attend.cuh"
#include "tree_merge.cuh"
#include "tree_scan.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// planner
// ---------------------------------------------------------------------------
constexpr int kTreePlanThreads = 1024;
constexpr int kTreePlanSmem = 2048;  // sequences whose prefix sums are searched in shared memory

// Cost of an item besides its steps, in steps: its queries, the pipeline that
// drains and fills again, its output.  Measured on 160 steps a CTA cut into 1
// to 16 items: 3 to 4 us an item of bf16 caches, 8 of one-byte ones (a step:
// 0.7 to 1.0, 1.3 to 1.7 us).  With 2 for all, ragged batches took 74 instead
// of 65 us (head_dim 64), 241 instead of 225 (INT8); 6 and 9 change nothing.
static int tree_item_steps(int kv_dtype, bool pair) { return pair ? 3 : kv_dtype == PKV_KV_BF16 ? 4 : 6; }

struct TreePlanArgs {
  const int32_t* context_lens;
  const int32_t* node_counts;  // NULL: T each
  int32_t* ctx_eff;            // [B] validated lengths
  long long* start;            // [B + 1] steps x KV heads before each sequence
  TreeBound* bounds;           // [max_shares + 1]
  int32_t* shares;
  __nv_bfloat16* out;
  unsigned* err;
  int B, T, Hkv, max_ctx, row_elems /* T * Hq * D */;
  int max_shares, min_steps, item_steps;
};

// CTA 0: lengths, the prefix sums of the sequences' steps, the shares'
// boundaries, zeros for inactive sequences.  Other CTAs: tree_scan_values.
//
// (Shares are equal in cost, tree_bound: with shares equal in steps a batch of
// short and long sequences left SMs idle for half the time.)
__global__ void __launch_bounds__(kTreePlanThreads) tree_plan_kernel(const TreePlanArgs a, const TreeScan scan) {
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x > 0) {  // block-uniform: these CTAs never reach the barriers below
    tree_scan_values(scan, (blockIdx.x - 1) * (blockDim.x / 32) + (threadIdx.x >> 5),
                     static_cast<int>(gridDim.x - 1) * (blockDim.x / 32));
    return;
  }
  __shared__ long long warp_tot[kTreePlanThreads / 32];
  __shared__ long long carry_s;
  __shared__ long long start_s[kTreePlanSmem + 1];
  __shared__ int ctx_s[kTreePlanSmem];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  if (tid == 0) carry_s = 0;
  __syncthreads();
  unsigned err = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    long long steps = 0;
    if (b < a.B) {
      int c = a.context_lens[b];
      const int nodes = a.node_counts != nullptr ? a.node_counts[b] : a.T;
      if (c < 0 || c > a.max_ctx) {
        err |= PKV_DEVERR_CONTEXT_LEN;
        c = 0;
      }
      if (nodes < 0 || nodes > a.T) {
        err |= PKV_DEVERR_TREE;
        c = 0;
      }
      if (nodes == 0) c = 0;  // every row is zero
      a.ctx_eff[b] = c;
      if (a.B <= kTreePlanSmem) ctx_s[b] = c;
      steps = tree_cost(c, a.item_steps, a.Hkv);
    }
    long long x = steps;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    if (warp == 0) {
      long long w = lane < threads / 32 ? warp_tot[lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += y;
      }
      warp_tot[lane] = w;
    }
    __syncthreads();
    const long long before = carry_s + (warp > 0 ? warp_tot[warp - 1] : 0) + x - steps;
    if (b < a.B) {
      a.start[b] = before;
      if (a.B <= kTreePlanSmem) start_s[b] = before;
    }
    __syncthreads();
    if (tid == 0) carry_s += warp_tot[31];
    __syncthreads();
  }
  if (err) atomicOr(a.err, err);
  const long long total = carry_s;
  if (tid == 0) {
    a.start[a.B] = total;
    if (a.B <= kTreePlanSmem) start_s[a.B] = total;
  }
  __syncthreads();
  const long long* start = a.B <= kTreePlanSmem ? start_s : a.start;
  const int shares = tree_share_count(total, a.min_steps, a.max_shares);
  if (tid == 0) *a.shares = shares;
#pragma unroll 1
  for (int s = tid; s <= shares; s += threads) {
    TreeBound r = tree_bound(s, shares, total, start, a.B, a.Hkv, a.item_steps);
    if (r.b < a.B) r.ctx = a.B <= kTreePlanSmem ? ctx_s[r.b] : a.ctx_eff[r.b];
    a.bounds[s] = r;
  }
  // zeros for inactive sequences (one warp per sequence)
#pragma unroll 1
  for (int b = warp; b < a.B; b += threads / 32) {
    if (start[b + 1] != start[b]) continue;
    uint4* o = reinterpret_cast<uint4*>(a.out + static_cast<size_t>(b) * a.row_elems);
#pragma unroll 1
    for (int i = lane; i < a.row_elems / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, int KV, bool PAIR>
static const void* attend_instance(int bs) {
  return bs == 16 ? reinterpret_cast<const void*>(&tree_attend_kernel<D, 16, KV, PAIR, false>)
                  : reinterpret_cast<const void*>(&tree_attend_kernel<D, 32, KV, PAIR, false>);
}

struct TreeKernel {
  const void* fn;
  size_t smem;
  int threads;
};
template <int D, int KV>
static TreeKernel attend_kernel(int bs, bool pair) {
  return pair ? TreeKernel{attend_instance<D, KV, true>(bs), TaLayout<D, KV, true>::kBytes, ta_threads(KV)}
              : TreeKernel{attend_instance<D, KV, false>(bs), TaLayout<D, KV, false>::kBytes, ta_threads(KV)};
}
static TreeKernel pick(int kv_dtype, int D, int bs, bool pair) {
  if (kv_dtype == PKV_KV_FP8_E4M3) return attend_kernel<128, PKV_KV_FP8_E4M3>(bs, pair);
  if (kv_dtype == PKV_KV_INT8) return attend_kernel<128, PKV_KV_INT8>(bs, pair);
  return D == 64 ? attend_kernel<64, PKV_KV_BF16>(bs, pair) : attend_kernel<128, PKV_KV_BF16>(bs, pair);
}

size_t tree_attend_smem_bytes(int kv_dtype, int D, int pair) { return pick(kv_dtype, D, 16, pair != 0).smem; }

static size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

TreeWorkspace tree_workspace(int B, int Hkv, int D, int NT, int tree_words, int max_shares) {
  const int NP = NT > 1 ? (NT + 1) / 2 : 1, tiles = NT > 1 ? 2 : 1;
  const size_t rows = static_cast<size_t>(max_shares) * NP * 2 * tiles * kTaRows;
  TreeWorkspace w{};
  size_t off = 0;
  w.shares = off;
  off += 256;
  w.ctx_eff = off;
  off = align_up(off + sizeof(int32_t) * static_cast<size_t>(B));
  w.start = off;
  off = align_up(off + sizeof(long long) * (static_cast<size_t>(B) + 1));
  w.bounds = off;
  off = align_up(off + sizeof(TreeBound) * (static_cast<size_t>(max_shares) + 1));
  w.poison = off;
  off = align_up(off + sizeof(uint32_t) * static_cast<size_t>(B) * Hkv * tree_words);
  w.part_ml = off;
  off = align_up(off + sizeof(float2) * rows);
  w.part_o = off;
  off = align_up(off + sizeof(float) * D * rows);
  w.total = off;
  return w;
}

// Raises a kernel's dynamic shared memory limit, once per (device, context,
// kernel); checks that it is launched with the registers that its warps share
// out (a warp that waits for more than there are would wait forever).
cudaError_t allow_smem(const void* fn, size_t smem, int regs) {
  struct Entry {
    int dev;
    void* ctx;
    const void* fn;
  };
  static std::mutex mu;
  static std::vector<Entry> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  void* ctx = current_context();
  std::lock_guard<std::mutex> lock(mu);
  for (const Entry& x : done)
    if (x.dev == dev && x.ctx == ctx && ctx != nullptr && x.fn == fn) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaFuncAttributes at{};
  e = cudaFuncGetAttributes(&at, fn);
  if (e != cudaSuccess) return e;
  if (at.numRegs != regs) return cudaErrorInvalidKernelImage;
  done.push_back(Entry{dev, current_context(), fn});
  return cudaSuccess;
}

cudaError_t launch_tree_attend(const DecodeLaunch& L, uint8_t* ws, int* launched) {
  const bool pair = L.NT > 1;
  const int NP = pair ? (L.NT + 1) / 2 : 1;
  const TreeKernel k = pick(L.kv_dtype, L.D, L.bs, pair);
  cudaError_t e = allow_smem(k.fn, k.smem, ta_launch_regs(L.kv_dtype));
  if (e != cudaSuccess) return e;
  const TreeWorkspace w = tree_workspace(L.B, L.Hkv, L.D, L.NT, L.tree_words, L.tree_shares);
  int32_t* shares = reinterpret_cast<int32_t*>(ws + w.shares);
  int32_t* ctx_eff = reinterpret_cast<int32_t*>(ws + w.ctx_eff);
  TreeBound* bounds = reinterpret_cast<TreeBound*>(ws + w.bounds);
  uint32_t* poison = reinterpret_cast<uint32_t*>(ws + w.poison);

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.stream = L.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;

  // 1. planner
  TreePlanArgs pa{L.context_lens, L.node_counts, ctx_eff, reinterpret_cast<long long*>(ws + w.start), bounds, shares,
                  static_cast<__nv_bfloat16*>(L.out), L.err, L.B, L.T, L.Hkv, L.MB * L.bs, L.T * L.Hq * L.D,
                  L.tree_shares, L.tree_min_steps, tree_item_steps(L.kv_dtype, pair)};
  const TreeScan scan = tree_scan_of(L, poison);
  // (a thread per share, or sequence: a CTA of 1024 takes longer to start)
  const int plan_threads = L.B <= 192 ? 192 : kTreePlanThreads;
  cfg.gridDim = dim3(1 + tree_scan_ctas(L, plan_threads / 32));
  cfg.blockDim = dim3(plan_threads);
  e = cudaLaunchKernelEx(&cfg, tree_plan_kernel, pa, scan);
  if (e != cudaSuccess) return e;
  *launched += 1;

  // 2. attention: one CTA per share and row-tile pair
  TaParams p{};
  p.q = static_cast<const __nv_bfloat16*>(L.q);
  p.out = static_cast<__nv_bfloat16*>(L.out);
  p.block_tables = L.block_tables;
  p.k_scale = L.k_scale;
  p.v_scale = L.v_scale;
  p.ctx_eff = ctx_eff;
  p.bounds = bounds;
  p.shares = shares;
  p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.err = L.err;
  p.tree.mask = L.tree_mask;
  p.tree.node_counts = L.node_counts;
  p.tree.poison = L.kv_dtype != PKV_KV_INT8 ? poison : nullptr;
  p.tree.words = L.tree_words;
  p.tree.stride = L.tree_stride;
  p.Hq = L.Hq;
  p.Hkv = L.Hkv;
  p.G = L.G;
  p.T = L.T;
  p.Tt = L.Tt;
  p.NT = L.NT;
  p.NP = NP;
  p.MB = L.MB;
  p.NB = L.NB;
  p.row_base = L.row_base;
  p.scale_log2 = L.scale_log2;
  CUtensorMap kmap = L.kmap, vmap = L.vmap, qmap = L.qmap;
  void* args[] = {&kmap, &vmap, &qmap, &p};
  cfg.gridDim = dim3(static_cast<unsigned>(L.tree_shares * NP));
  cfg.blockDim = dim3(k.threads);
  cfg.dynamicSmemBytes = k.smem;
  cfg.numAttrs = (L.ev_start == nullptr) ? 1 : 0;  // an event between them: no overlap with the planner
  if (L.ev_start != nullptr && (e = cudaEventRecord(L.ev_start, L.stream)) != cudaSuccess) return e;
  e = cudaLaunchKernelExC(&cfg, k.fn, args);
  if (e != cudaSuccess) return e;
  if (L.ev_end != nullptr && (e = cudaEventRecord(L.ev_end, L.stream)) != cudaSuccess) return e;
  *launched += 1;

  // 3. merge of the items that shares split
  if (L.tree_shares > 1) {
    const TreeMergeArgs ma{bounds, nullptr, shares, p.part_ml, p.part_o, p.out, L.Hq, L.G, L.T, L.Tt, NP, pair ? 2 : 1};
    cfg.gridDim = dim3(static_cast<unsigned>((L.tree_shares - 1) * NP * (ma.tiles * kTaRows / merge_cta_rows(2))));
    cfg.blockDim = dim3(kTreeMergeThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = (L.ev_end == nullptr) ? 1 : 0;
    e = L.D == 64 ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<64, false, 2>, ma) : cudaLaunchKernelEx(&cfg, tree_merge_kernel<128, false, 2>, ma);
    if (e != cudaSuccess) return e;
    *launched += 1;
  }
  return cudaSuccess;
}

}  // namespace pkv
