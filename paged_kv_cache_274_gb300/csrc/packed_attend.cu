// Planner and launch of the tcgen05 attention of packed rows (tree_attend.cuh
// with PACKED), and its kernel instances.
//
// Sequence b's rows are consecutive rows of q and out; row t of m sees the
// positions up to ctx - m + t.  The rows of a KV head form tiles of 128 (row,
// head) rows; the kernel steps through the positions that a tile (or a pair of
// tiles) sees, 128 at a time, and masks the last steps row by row.
#include <algorithm>

#include "tree_merge.cuh"
#include "tree_scan.cuh"

namespace pkv {

constexpr int kPackedPlanThreads = 1024;
constexpr int kPackedPlanSmem = 1024;  // sequences whose sums are searched in shared memory

// Cost of an item besides its steps, in steps (tree_attend.cu), measured for pairs
// of tiles on three batches of each kind (us): head_dim 64 5 (ragged prompts 146, 138,
// 168; 3: 149, 143, 171; 4: 145, 144, 170; 8: 148, 140, 169), one byte 6 (E4M3 359, 247,
// 271; 2: 406, 279, 315; 4: 362, 246, 272; 8: 366, 250, 277; INT8 82, 104, 90; 3: 83, 99,
// 92; 8: 84, 103, 91), bf16 4, where nothing stands out (a prompt of 8192 tokens 428 to
// 447 in one loop, with 2 437, 3 446 to 459, 5 444 to 447, 8 453; chunks beside single
// tokens 2 to 8 within 3%).
static int packed_item_steps(int kv_dtype, int D, bool pair) {
  if (kv_dtype == PKV_KV_BF16) return pair && D == 64 ? 5 : 4;
  return 6;
}

// What a step of an item with one row tile costs where CTAs serve pairs of
// tiles, of kPackedWeight (chunks of prompts beside single tokens, three batches, us:
// bf16 6: 311 to 331, 378, 395; 5: 313, 368, 391; 4: 329, 402, 422; 8: 358, 407, 432;
// E4M3 5: 360, 248, 272; 4: 389, 270, 294; 6: 362, 249, 274; INT8 5: 82, 104, 89; 4: 81,
// 96, 86; 6: 86, 105, 97).
static int packed_alone(int kv_dtype) { return kv_dtype == PKV_KV_BF16 ? 6 : 5; }

struct PackedPlanArgs {
  const int32_t* context_lens;
  const int32_t* query_starts;
  const int32_t* block_tables;
  const uint8_t* v;   // the cache slot's V pages
  PackedSeq* seqs;    // [B]
  long long* start;   // [B + 1]
  PackedBound* bounds;
  int32_t* shares;
  uint32_t* poison;   // [Hkv][words] rows whose V is not finite; NULL: INT8
  __nv_bfloat16* out;
  unsigned* err;
  int B, N, T, Hkv, MB, NB, bs, words, row_bytes, e4m3;
  int span, tile, alone, max_shares, min_steps, item_steps, row_elems /* Hq * D */;
};

// A sequence as the caller gives it.
struct PackedGiven {
  int s0, s1, ctx;
};
__device__ __forceinline__ PackedGiven packed_given(const PackedPlanArgs& a, int b) {
  return b < a.B ? PackedGiven{a.query_starts[b], a.query_starts[b + 1], a.context_lens[b]} : PackedGiven{0, 0, 0};
}

// The first sequence whose entries of query_starts fall, or B.  The whole CTA;
// a barrier.  (`own`: this thread's first sequence, loaded before it.)
__device__ __forceinline__ int packed_first_fall(const PackedPlanArgs& a, const PackedGiven& own) {
  __shared__ int fall_s;
  int mine = own.s1 < own.s0 ? static_cast<int>(threadIdx.x) : a.B;
#pragma unroll 1
  for (int b = threadIdx.x + blockDim.x; b < a.B && mine == a.B; b += blockDim.x)
    if (packed_falls(a.query_starts, b)) mine = b;
  if (threadIdx.x == 0) fall_s = a.B;
  if (!__syncthreads_or(mine < a.B)) return a.B;
  atomicMin(&fall_s, mine);
  __syncthreads();
  return fall_s;
}

// Sequence b, checked.
__device__ __forceinline__ PackedSeq packed_seq(const PackedPlanArgs& a, const PackedGiven& x, int b, int fall, unsigned& err) {
  const int s0 = x.s0, s1 = x.s1;
  int c = x.ctx, m = 0;
  if (packed_rows_fit(s0, s1, b, fall, a.N, a.T))
    m = s1 - s0;
  else
    err |= PKV_DEVERR_QUERY;
  if (c < 0 || c > a.MB * a.bs) {
    err |= PKV_DEVERR_CONTEXT_LEN;
    c = 0;
  }
  return PackedSeq{c, m > 0 ? s0 : 0, m, 0};
}

// Rows' words warp0, warp0 + nwarps, ...: zeros for the rows that see nothing
// (with the first KV head's words), and which V rows are not finite: those
// would reach every row of a tile through 0 x NaN, so the attention leaves them
// out of the products and sets the rows that see them to NaN (tree_scan.cuh).
__device__ __forceinline__ void packed_scan(const PackedPlanArgs& a, int fall, int warp0, int nwarps) {
  const int lane = threadIdx.x & 31;
  const int heads = a.poison != nullptr ? a.Hkv : 1;
#pragma unroll 1
  for (int i = warp0; i < heads * a.words; i += nwarps) {  // (less than 2^31, as the host checks)
    const int h = i / a.words, w = i - h * a.words, row = 32 * w + lane;
    bool zero = false;
    long long at = -1;
    if (row < a.N) {
      const int b = packed_owner(a.query_starts, fall, row);
      if (b >= 0) {
        unsigned err = 0;  // (the planner reports it)
        const PackedSeq s = packed_seq(a, packed_given(a, b), b, fall, err);
        const int t = row - s.start, pos = s.ctx - s.m + t;
        if (t < s.m) {
          zero = pos < 0;
          // (a sequence's first row is seen by all others)
          if (pos >= 0 && t > 0 && a.poison != nullptr) {
            const int blk = __ldg(a.block_tables + static_cast<size_t>(b) * a.MB + pos / a.bs);
            if (static_cast<unsigned>(blk) < static_cast<unsigned>(a.NB))
              at = ((static_cast<long long>(blk) * a.Hkv + h) * a.bs + pos % a.bs) * a.row_bytes;
          }
        }
      }
    }
    if (a.poison != nullptr) {
      uint32_t word = 0u;
      if (__any_sync(kFull, at >= 0)) word = a.row_bytes == 256 ? scan_rows<16>(a.v, at, a.e4m3 != 0) : scan_rows<8>(a.v, at, a.e4m3 != 0);
      if (lane == 0) a.poison[i] = word;
    }
    unsigned zeros = h == 0 ? __ballot_sync(kFull, zero) : 0u;
#pragma unroll 1
    for (; zeros != 0; zeros &= zeros - 1) {
      uint4* o = reinterpret_cast<uint4*>(a.out + static_cast<size_t>(32 * w + __ffs(zeros) - 1) * a.row_elems);
#pragma unroll 1
      for (int k = lane; k < a.row_elems / 8; k += 32) o[k] = make_uint4(0, 0, 0, 0);
    }
  }
}

// CTA 0: the sequences, the prefix sums of their costs, the shares' boundaries.
// Other CTAs: packed_scan.
__global__ void __launch_bounds__(kPackedPlanThreads) packed_plan_kernel(const PackedPlanArgs a) {
  pdl_trigger();
  pdl_wait();
  __shared__ long long carry_s;
  if (threadIdx.x == 0) carry_s = 0;
  PackedGiven given = packed_given(a, threadIdx.x);
  const int fall = packed_first_fall(a, given);
  if (blockIdx.x > 0) {  // block-uniform: these CTAs never reach the barriers below
    packed_scan(a, fall, (blockIdx.x - 1) * (blockDim.x / 32) + (threadIdx.x >> 5), static_cast<int>(gridDim.x - 1) * (blockDim.x / 32));
    return;
  }
  __shared__ long long warp_tot[kPackedPlanThreads / 32];
  __shared__ long long start_s[kPackedPlanSmem + 1];
  __shared__ PackedSeq seq_s[kPackedPlanSmem];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const bool fits = a.B <= kPackedPlanSmem;
  const long long item_cost = packed_item_cost(a.item_steps);
  unsigned err = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += threads) {
    const int b = b0 + tid;
    long long cost = 0;
    if (b0 > 0) given = packed_given(a, b);
    if (b < a.B) {
      const PackedSeq s = packed_seq(a, given, b, fall, err);
      a.seqs[b] = s;
      if (fits) seq_s[b] = s;
      cost = packed_cost(s, a.span, item_cost) * packed_weight(s, a.tile, a.alone) * a.Hkv;
    }
    long long x = cost;
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
    const long long before = carry_s + (warp > 0 ? warp_tot[warp - 1] : 0) + x - cost;
    if (b < a.B) {
      a.start[b] = before;
      if (fits) start_s[b] = before;
    }
    __syncthreads();
    if (tid == 0) carry_s += warp_tot[31];
    __syncthreads();
  }
  if (err) atomicOr(a.err, err);
  const long long total = carry_s;
  if (tid == 0) {
    a.start[a.B] = total;
    if (fits) start_s[a.B] = total;
  }
  __syncthreads();
  const int shares = packed_share_count(total, a.min_steps, a.max_shares);
  if (tid == 0) *a.shares = shares;
#pragma unroll 1
  for (int s = tid; s <= shares; s += threads)
    a.bounds[s] = packed_bound(s, shares, total, fits ? start_s : a.start, fits ? seq_s : a.seqs, a.B, a.Hkv, a.span, a.tile, a.alone, a.item_steps);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, int KV, bool PAIR>
static const void* packed_instance(int bs) {
  return bs == 16 ? reinterpret_cast<const void*>(&tree_attend_kernel<D, 16, KV, PAIR, true>)
                  : reinterpret_cast<const void*>(&tree_attend_kernel<D, 32, KV, PAIR, true>);
}

struct PackedKernel {
  const void* fn;
  size_t smem;
};
template <int D, int KV>
static PackedKernel packed_kernel(int bs, bool pair) {
  return pair ? PackedKernel{packed_instance<D, KV, true>(bs), TaLayout<D, KV, true>::kBytes}
              : PackedKernel{packed_instance<D, KV, false>(bs), TaLayout<D, KV, false>::kBytes};
}
static PackedKernel packed_pick(int kv_dtype, int D, int bs, bool pair) {
  if (kv_dtype == PKV_KV_FP8_E4M3) return packed_kernel<128, PKV_KV_FP8_E4M3>(bs, pair);
  if (kv_dtype == PKV_KV_INT8) return packed_kernel<128, PKV_KV_INT8>(bs, pair);
  return D == 64 ? packed_kernel<64, PKV_KV_BF16>(bs, pair) : packed_kernel<128, PKV_KV_BF16>(bs, pair);
}

PackedWorkspace packed_workspace(int B, int N, int Hkv, int D, int tiles, int max_shares) {
  const size_t rows = static_cast<size_t>(max_shares) * 2 * tiles * kTaRows;
  PackedWorkspace w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  w.shares = take(4);
  w.seqs = take(sizeof(PackedSeq) * static_cast<size_t>(B));
  w.start = take(sizeof(long long) * (static_cast<size_t>(B) + 1));
  w.bounds = take(sizeof(PackedBound) * (static_cast<size_t>(max_shares) + 1));
  w.merge = take(sizeof(PackedMerge) * static_cast<size_t>(max_shares));
  w.poison = take(sizeof(uint32_t) * static_cast<size_t>(Hkv) * ((static_cast<size_t>(N) + 31) / 32));
  w.part_ml = take(sizeof(float2) * rows);
  w.part_o = take(sizeof(float) * D * rows);
  w.total = off;
  return w;
}

cudaError_t launch_packed_attend(const DecodeLaunch& L, uint8_t* ws, int* launched) {
  const bool pair = L.NT > 1;
  const int tiles = pair ? 2 : 1, words = (L.N + 31) / 32;
  const PackedKernel k = packed_pick(L.kv_dtype, L.D, L.bs, pair);
  cudaError_t e = allow_smem(k.fn, k.smem, ta_launch_regs(L.kv_dtype));
  if (e != cudaSuccess) return e;
  const PackedWorkspace w = packed_workspace(L.B, L.N, L.Hkv, L.D, tiles, L.tree_shares);
  int32_t* shares = reinterpret_cast<int32_t*>(ws + w.shares);
  PackedSeq* seqs = reinterpret_cast<PackedSeq*>(ws + w.seqs);
  PackedBound* bounds = reinterpret_cast<PackedBound*>(ws + w.bounds);
  uint32_t* poison = L.kv_dtype != PKV_KV_INT8 ? reinterpret_cast<uint32_t*>(ws + w.poison) : nullptr;

  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.stream = L.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;

  // 1. planner, with a warp per word of rows up to a full GPU
  const PackedPlanArgs pa{L.context_lens, L.query_starts, L.block_tables, static_cast<const uint8_t*>(L.v_cache), seqs,
                          reinterpret_cast<long long*>(ws + w.start), bounds, shares, poison, static_cast<__nv_bfloat16*>(L.out), L.err,
                          L.B, L.N, L.T, L.Hkv, L.MB, L.NB, L.bs, words, L.D * (L.kv_fp8 ? 1 : 2), L.kv_dtype == PKV_KV_FP8_E4M3 ? 1 : 0,
                          tiles * L.Tt, L.Tt, pair ? packed_alone(L.kv_dtype) : kPackedWeight, L.tree_shares, L.tree_min_steps, packed_item_steps(L.kv_dtype, L.D, pair), L.Hq * L.D};
  const int plan_threads = L.B <= 192 ? 192 : kPackedPlanThreads;
  const long long scans = static_cast<long long>(poison != nullptr ? L.Hkv : 1) * words;
  const int warps = plan_threads / 32;
  cfg.gridDim = dim3(static_cast<unsigned>(1 + std::min<long long>((scans + warps - 1) / warps, 151 * 32 / warps)));
  cfg.blockDim = dim3(plan_threads);
  e = cudaLaunchKernelEx(&cfg, packed_plan_kernel, pa);
  if (e != cudaSuccess) return e;
  *launched += 1;

  // 2. attention: one CTA per share
  TaParams p{};
  p.q = static_cast<const __nv_bfloat16*>(L.q);
  p.out = static_cast<__nv_bfloat16*>(L.out);
  p.block_tables = L.block_tables;
  p.k_scale = L.k_scale;
  p.v_scale = L.v_scale;
  p.shares = shares;
  p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.err = L.err;
  p.tree.poison = poison;
  p.tree.words = words;
  p.Hq = L.Hq;
  p.Hkv = L.Hkv;
  p.G = L.G;
  p.T = L.T;
  p.Tt = L.Tt;
  p.NT = L.NT;
  p.NP = 1;
  p.MB = L.MB;
  p.NB = L.NB;
  p.row_base = L.row_base;
  p.scale_log2 = L.scale_log2;
  p.seqs = seqs;
  p.pbounds = bounds;
  p.merge = reinterpret_cast<PackedMerge*>(ws + w.merge);
  CUtensorMap kmap = L.kmap, vmap = L.vmap, qmap = L.qmap;
  void* args[] = {&kmap, &vmap, &qmap, &p};
  cfg.gridDim = dim3(static_cast<unsigned>(L.tree_shares));
  cfg.blockDim = dim3(ta_threads(L.kv_dtype));
  cfg.dynamicSmemBytes = k.smem;
  cfg.numAttrs = (L.ev_start == nullptr) ? 1 : 0;  // an event between them: no overlap with the planner
  if (L.ev_start != nullptr && (e = cudaEventRecord(L.ev_start, L.stream)) != cudaSuccess) return e;
  e = cudaLaunchKernelExC(&cfg, k.fn, args);
  if (e != cudaSuccess) return e;
  if (L.ev_end != nullptr && (e = cudaEventRecord(L.ev_end, L.stream)) != cudaSuccess) return e;
  *launched += 1;

  // 3. merge of the items that shares split
  if (L.tree_shares > 1) {
    const TreeMergeArgs ma{nullptr, p.merge, shares, p.part_ml, p.part_o, p.out, L.Hq, L.G, L.T, L.Tt, 1, tiles};
    cfg.gridDim = dim3(static_cast<unsigned>((L.tree_shares - 1) * (tiles * kTaRows / merge_cta_rows(2 * tiles))));
    cfg.blockDim = dim3(kTreeMergeThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = (L.ev_end == nullptr) ? 1 : 0;
    auto merge = pair ? (L.D == 64 ? tree_merge_kernel<64, true, 4> : tree_merge_kernel<128, true, 4>)
                      : (L.D == 64 ? tree_merge_kernel<64, true, 2> : tree_merge_kernel<128, true, 2>);
    e = cudaLaunchKernelEx(&cfg, merge, ma);
    if (e != cudaSuccess) return e;
    *launched += 1;
  }
  return cudaSuccess;
}

}  // namespace pkv
