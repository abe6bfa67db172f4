// Attention of drafted-tree nodes over the paged cache on the 5th-generation
// tensor cores (tcgen05 + TMEM): bf16 caches of head_dim 64 and 128, E4M3 and
// INT8 caches of head_dim 128.
//
// A sequence of n cached tokens whose last m are tree nodes has T x G (node,
// head) rows per KV head; row t attends to the base = n - m tokens before the
// tree and to the nodes of its mask row (tree_mask.cuh).  The rows form tiles
// of 128 (M of the MMA); the cache is stepped through 128 tokens at a time.
//
// What bounds it: with one tile of rows the cache bytes, 64 KiB (bf16, D 128)
// or 32 KiB (one byte) per 128 tokens of one KV head, 1.47 or 0.73 us of an
// SM's share of the measured HBM rate, next to 0.67 us of tensor pipe (at the
// measured bf16 rate) for S = Q K^T and O += P V; with two tiles the tensor
// pipe, 1.34 us.  Measured per step of 128 tokens with the cache in L2: bf16
// 0.87 to 1.0 us with one tile, 1.65 with two (D 64: 0.70 to 0.76, 1.42), E4M3
// 1.15 to 1.35 and 2.3, INT8 1.65 to 1.75 and 2.7.  So bf16 batches of one tile
// run at HBM speed (64 sequences of 2048 to 4096 tokens, 32 nodes, 8 KV heads:
// 156 us with plan and merge, 0.80 of the copy rate), long contexts with many
// rows at 0.64 of the bf16 peak (4 x 32k tokens, 64 nodes, 8 heads a KV head:
// 218 us).  One-byte caches fill no unit: a sub-partition issues 1600
// instructions a step, against 940 of bf16 caches, for the page scales and the
// widening, but only 60% (E4M3) or 53% (INT8) of the time, with DRAM at 41 and
// 29% and the tensor pipe at 38 and 27%: a step is a chain of hand-overs (codes
// landed, widened, S, the maximum agreed, P, PV).
//
// One CTA per SM, no CTA-wide barrier inside the loop:
//   * Two streams of eight softmax warps, each stream with its own S and O in
//     tensor memory (S0 S1 O0 O1, 128 columns each), so that the products of
//     one run while the other's softmax does.  Two warps share 32 rows, one
//     half of the step's tokens each: a row's exponentials then take half as
//     long between S and PV (one warp per 32 rows: 90 instead of 79 us for the
//     D 64 batch).  PAIR: the streams hold two row tiles of one KV head and
//     read every step of the cache together.  Otherwise there is one row tile,
//     stream 0 takes the even steps and stream 1 the odd ones, and a work unit
//     ends with the sum of the two (as split-K partials would be joined).
//   * One thread issues, step after step, PV_i of the stream's step before and
//     S_i of this one; P (16 bits) overwrites the S columns it came from and is
//     the A operand of PV.  tcgen05 operations of one thread complete in order,
//     so S_i never overwrites a P_i that is still read.  (Measured and left:
//     three S buffers with one O, 0.95 instead of 0.87 us a step; PV of the
//     first 32 tokens of each half while the others' P is made, 1.71 instead
//     of 1.65 for two tiles.)
//   * A K copy warp walks the CTA's share of the work, publishes a descriptor
//     per step (page ids, page parameters) in a ring, and copies K pages; a V
//     copy warp copies V pages; for bf16 caches a query warp the query tiles.
//   * One-byte caches add eight converter warps: they rewrite V pages (and INT8
//     K pages) in their stage as exact 16-bit code values, and the query rows
//     in the type of the K operand (E4M3 K pages feed the products as they
//     are, against a query of two E4M3 parts).  Four of them took 2.25 instead
//     of 1.68 us an INT8 step.  The page scales multiply the scores and P.
//
// Work split ("stream-K"): the steps of all (sequence, KV head) items in a row
// are cut into equal shares, one per SM, whatever the lengths; a share that
// starts or ends inside an item leaves partials (m, l, O) for the merge
// kernel, at most two per CTA.  Boundaries near an item's ends move there.
// The shares depend on the lengths only, so results do not vary between runs.
//
// The running maximum is lazy (moved when it grows by more than 2^8), so O is
// rarely rescaled.  S, m, l and O are fp32; P is rounded to bf16 (bf16 caches:
// both operands of a product have one type) or f16 (one-byte caches).  Every
// wait is bounded; a CTA that gives up records PKV_DEVERR_TIMEOUT, lets its own
// copies and products finish (bounded) and frees its tensor memory.
#pragma once

#include <cstddef>

#include "paged_decode_tc2.cuh"
#include "tree_plan.cuh"

namespace pkv {

constexpr int kTaRows = 128;    // query rows per tile
constexpr int kTaRing = 8;      // step descriptors: a step's is read until its softmax is done, at most 5 steps back
constexpr uint32_t kTaCols = 512;  // TMEM: S0 0, S1 128, O0 256, O1 384

struct TaParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* block_tables;
  const float* k_scale;
  const float* v_scale;
  const int32_t* ctx_eff;
  const TreeBound* bounds;  // [shares + 1]
  const int32_t* shares;    // number of shares in use
  float2* part_ml;          // [CTA][2][tiles per CTA x 128]
  float* part_o;            // [CTA][2][tiles per CTA x 128][D]
  unsigned* err;
  TreeArgs tree;
  int Hq, Hkv, G, T, Tt, NT, NP, MB, NB, row_base;
  float scale_log2;
};

// Step flags; a step without any is every row's in whole, with scores whose
// order the page scales keep.
constexpr int kStepMasked = 1;  // the sequence's end, nodes, or a bad page
constexpr int kStepScales = 2;  // a k scale < 0, a v scale <= 0, or one that is not finite

// One step's descriptor in the ring.
struct TaStep {
  int n;      // steps of the work unit (0: no more work)
  int b, kvh;
  int t0, t1;  // the unit's tokens
  int part;    // 0: the unit is its whole item; else 1 + index of the CTA's partial
  int np;      // pages of this step
  int ctx;
  int pages[8];
  uint8_t bad[8];   // page id out of range
  int flags;        // kStepMasked, kStepScales
  float vref;       // one-byte caches: P carries v scale / vref
  // one-byte caches, per page: k scale, INT8 K bias 1152 + zero, v scale /
  // vref and its log2
  float4 par[8];
  float vzero[8];   // INT8: V zero point
};

// 16 softmax warps, the issuing, K copy, V copy and query warps, and for
// one-byte caches the converter warps
constexpr int kConvWarps = 8;
__host__ __device__ constexpr int ta_threads(int kv) { return kv == PKV_KV_BF16 ? 640 : 640 + 32 * kConvWarps; }
// Registers a thread at the launch (65,536 / threads, a multiple of 8), and
// after the warps have shared them out.
__host__ __device__ constexpr int ta_launch_regs(int kv) { return kv == PKV_KV_BF16 ? 96 : 72; }
__host__ __device__ constexpr int ta_role_regs(int kv) { return kv == PKV_KV_BF16 ? 48 : 40; }
__host__ __device__ constexpr int ta_soft_regs(int kv) {
  return (ta_threads(kv) * ta_launch_regs(kv) - (ta_threads(kv) - 512) * ta_role_regs(kv)) / 512 / 8 * 8;
}
static_assert(ta_soft_regs(PKV_KV_BF16) == 104 && ta_soft_regs(PKV_KV_INT8) == 96, "");

template <int D, int KV, bool PAIR>
struct TaLayout {  // byte offsets from the 1024-aligned shared-memory base
  static constexpr bool kOneByte = KV != PKV_KV_BF16;
  static constexpr bool kF8K = KV == PKV_KV_FP8_E4M3;
  static constexpr uint32_t kRegion = kTreeTokens * 128;      // 128 rows of 128 bytes
  static constexpr uint32_t kTile = (D / 64) * kRegion;       // 128 rows of D 16-bit values
  static constexpr uint32_t kKTile = kF8K ? kRegion : kTile;  // E4M3 K: codes
  static constexpr int kQTiles = PAIR ? 2 : 1;
  // stages: as many as fit beside the query tiles
  static constexpr int kKStages = D == 64 ? 4 : kF8K ? (PAIR ? 3 : 4) : PAIR ? 2 : 3;
  static constexpr int kVStages = D == 64 ? 4 : (kF8K && !PAIR) ? 3 : 2;
  static constexpr uint32_t kQ = 0;  // E4M3: the two parts of a tile, kRegion each
  static constexpr uint32_t kK = kQ + kQTiles * kTile;
  static constexpr uint32_t kV = kK + kKStages * kKTile;
  static constexpr uint32_t kBars = kV + kVStages * kTile;
  // k_full k_free tma_k [K], v_full v_free tma_v [V], s_full p_full o_full
  // o_free [2], step_full [ring], q_full q_free q_read x_full mma_drain
  static constexpr int kNumBars = 3 * kKStages + 3 * kVStages + 8 + kTaRing + 5;
  static constexpr uint32_t kMisc = kBars + 8 * kNumBars;
  static constexpr uint32_t kRing = (kMisc + 4 + 15) & ~15u;
  static constexpr uint32_t kStep = kOneByte ? sizeof(TaStep) : offsetof(TaStep, par);
  // exchanged among the softmax warps: [stream][half][128] maxima (a pair's
  // streams: sums too); one tile: [stream][half][128] sums, [stream][128] m,
  // [stream] vref, apart because a stream may be in the next unit already
  static constexpr uint32_t kXml = kRing + kTaRing * kStep;
  static constexpr uint32_t kQrow = kXml + 4 * kTaRows * 4 + (PAIR ? 0 : 6 * kTaRows * 4 + 16);
  // one-byte caches: (2^kq, sum of q) per query row
  static constexpr uint32_t kEnd = kQrow + (kOneByte ? kQTiles * kTaRows * 8 : 0);
  static constexpr size_t kBytes = 1024 + kEnd;
  static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
  static_assert(sizeof(TaStep) % 16 == 0 && offsetof(TaStep, par) % 16 == 0, "");
};

// D[tmem] (+)= A[smem] . B[smem]^T with E4M3 operands (kind::f8f6f4); one thread.
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u));
}

// Waits for phase `parity` of `bar`; false after about two seconds.  Few
// instructions, because the kernel has some forty of these: the hardware
// suspends the thread for up to a microsecond per try.
constexpr int kTaTries = 1 << 21;
constexpr int kConvTries = 1 << 24;  // of 100 ns and more
__device__ __forceinline__ bool ta_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_addr(bar);
#pragma unroll 1
  for (int n = 0; n < kTaTries; ++n) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}

// One lane of the converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// Barrier of `threads` threads (whole warps) on hardware barrier `id`; true if
// any of them says so.
__device__ __forceinline__ bool bar_red_or(int id, int threads, bool any) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(any ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Whole warp: 8 registers to consecutive TMEM columns, 16 from them.
__device__ __forceinline__ void tc_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_regs_loaded16(uint32_t (&v)[16]) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Largest of 16 scores (bit patterns of floats) from x[o] on.
__device__ __forceinline__ float max16(const uint32_t (&x)[32], int o) {
  auto f = [&](int i) { return __uint_as_float(x[o + i]); };
  const float a = fmax3f(f(0), f(1), f(2)), b = fmax3f(f(3), f(4), f(5)), c = fmax3f(f(6), f(7), f(8));
  const float d = fmax3f(f(9), f(10), f(11)), e = fmax3f(f(12), f(13), f(14));
  return fmax3f(fmax3f(a, b, c), fmax3f(d, e, f(15)), a);
}

// Rewrite 16 token rows of a stage whose one-byte codes lie in the upper half
// (row r's 128 codes at region + 128 r) as 16-bit code values in both halves
// (16-byte chunks XOR-swizzled by row % 8).  Whole warp: lanes 0-15 take codes
// 0-63 of a row each, which go to the lower half, the others codes 64-127; the
// warp reads all of its codes before it writes.
template <int KV, bool kBiased>
__device__ __forceinline__ void widen_rows(uint8_t* stage, uint32_t region, int lane, uint32_t zc, int valid_rows) {
  const int row = lane & 15, half = lane >> 4, sw = row & 7;
  const uint8_t* from = stage + region + row * 128;
  uint8_t* to = stage + half * region + row * 128;
  uint4 x[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) x[c] = *reinterpret_cast<const uint4*>(from + (((4 * half + c) ^ sw) << 4));
  __syncwarp();
  if (row < valid_rows) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 o0, o1;
      widen16<KV, kBiased>(x[c], zc, o0, o1);
      *reinterpret_cast<uint4*>(to + (((2 * c) ^ sw) << 4)) = o0;
      *reinterpret_cast<uint4*>(to + (((2 * c + 1) ^ sw) << 4)) = o1;
    }
  }
}

template <int D, int BS, int KV, bool PAIR>
__global__ void __launch_bounds__(ta_threads(KV), 1)
    tree_attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ CUtensorMap qmap,  // bf16: q [B][T][Hq][D], box 64 x G x Tt
                       const TaParams p) {
  using L = TaLayout<D, KV, PAIR>;
  constexpr bool kOneByte = L::kOneByte, kF8K = L::kF8K, kI8 = KV == PKV_KV_INT8;
  static_assert(!kOneByte || D == 128, "one-byte pages need head_dim 128");
  constexpr int PPI = kTreeTokens / BS;  // pages per step
  constexpr int KS = L::kKStages, VS = L::kVStages;
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // Barrier phases: k_* and v_* rings by the CTA's running step index g (stage
  // g % stages), step_full by g % ring; s_full and p_full once per step of a
  // stream; q_full, q_free, q_read, o_free, x_full once per unit; o_full[1] once per
  // unit with a step for stream 1.  Each barrier's next use depends on the wait
  // for its previous phase, so no waiter is ever two phases behind.
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + L::kBars);  // K of the step ready for the products
  uint64_t* k_free = k_full + KS;   // the step's S done
  uint64_t* tma_k = k_free + KS;    // INT8: K codes landed
  uint64_t* v_full = tma_k + KS;
  uint64_t* v_free = v_full + VS;   // the step's PV done
  uint64_t* tma_v = v_free + VS;    // one-byte: V codes landed
  uint64_t* s_full = tma_v + VS;    // [stream] S_i (and every product before it) done
  uint64_t* p_full = s_full + 2;    // [stream] P_i in TMEM, stale V rows cleared
  uint64_t* o_full = p_full + 2;    // [stream] the unit's last PV_i done
  uint64_t* o_free = o_full + 2;    // [stream] the unit's O_i read
  uint64_t* step_full = o_free + 2; // [ring] descriptor written
  uint64_t* q_full = step_full + kTaRing;
  uint64_t* q_free = q_full + 1;    // the unit's last S done
  uint64_t* q_read = q_free + 1;    // one-byte: the unit's row factors read by every softmax warp
  uint64_t* x_full = q_read + 1;    // one tile: both streams' (m, l) written
  uint64_t* mma_drain = x_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], kI8 ? kConvWarps : 1);
      mbar_init(&k_free[s], 1);
      mbar_init(&tma_k[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&v_full[s], kOneByte ? kConvWarps : 1);
      mbar_init(&v_free[s], 1);
      mbar_init(&tma_v[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 8);  // one lane per warp of the stream
      mbar_init(&o_full[s], 1);
      mbar_init(&o_free[s], PAIR ? 8 : 16);
    }
    for (int s = 0; s < kTaRing; ++s) mbar_init(&step_full[s], 1);
    mbar_init(q_full, kOneByte ? kConvWarps : 1);
    mbar_init(q_free, 1);
    mbar_init(q_read, 16);
    mbar_init(x_full, 16);
    mbar_init(mma_drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    if (!kOneByte) prefetch_tensormap(&qmap);
  }
  if (warp == 0) tc_alloc(tmem_slot, kTaCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  const int share = blockIdx.x / p.NP, pair = blockIdx.x - share * p.NP;
  bool timed_out = false;
  uint32_t k_issued = 0, v_issued = 0, q_loads = 0, mma_issued = 0;  // for the drain after a timeout

  auto step_at = [&](uint32_t g) { return reinterpret_cast<volatile TaStep*>(sm + L::kRing + (g % kTaRing) * L::kStep); };
  // this warp waits (lane 0, bounded) for phase `parity` of `bar`; false on timeout
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    int ok = 1;
    if (lane == 0) ok = ta_wait(bar, parity) ? 1 : 0;
    return __shfl_sync(kFull, ok, 0) != 0;
  };
  auto wait_step = [&](uint32_t g) { return warp_wait(&step_full[g % kTaRing], (g / kTaRing) & 1u); };

  // the registers are shared out anew: 512 x ta_soft_regs for the softmax
  // warps and the others' ta_role_regs add up to the launch's
  if (warp >= 16 && warp < 20) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ta_role_regs(KV)));
  if (warp == 17) {
    // K copy warp: the share's units, a descriptor and the K pages per step
    uint32_t g = 0;
    TreeBound at{0, 0, 0, 0}, end{0, 0, 0, 0};
    {  // (loaded side by side: every share has its place)
      const int shares = __ldg(p.shares);
      const TreeBound b0 = p.bounds[share], b1 = p.bounds[share + 1];
      if (share < shares) {
        at = b0;
        end = b1;
      }
    }
    int b = at.b, kvh = at.kvh, j0 = at.step;
    const uint64_t policy = p.NP > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    bool first_unit = true;
    float vref = 0.f;
    while (!timed_out && (b < end.b || (b == end.b && (kvh < end.kvh || (kvh == end.kvh && j0 < end.step))))) {
      const int ctx = b == at.b ? at.ctx : __ldg(p.ctx_eff + b);
      const int nt = (ctx + kTreeTokens - 1) / kTreeTokens;
      if (nt == 0) {  // an inactive sequence
        ++b;
        continue;
      }
      const int n = (b == end.b && kvh == end.kvh ? end.step : nt) - j0;
      const int t0 = j0 * kTreeTokens, t1 = min(ctx, (j0 + n) * kTreeTokens);
      const int part = tree_unit_part(j0, n, nt, first_unit);
      first_unit = false;
      vref = 0.f;  // of the unit; 0: no page with a scale yet
      const int npages = (t1 - t0 + BS - 1) / BS;
      const int base = ctx - (p.tree.node_counts != nullptr ? __ldg(p.tree.node_counts + b) : p.T);
      const int* trow = p.block_tables + static_cast<size_t>(b) * p.MB + t0 / BS;
      if constexpr (kOneByte) {  // the unit's queries, which the converters read once the unit before is done
        const int lines = 2 * p.G;
#pragma unroll 1
        for (int x = lane; x < L::kQTiles * p.Tt * lines; x += 32) {
          const int t = 2 * pair * p.Tt + x / lines;
          if (t < p.T)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + (static_cast<size_t>(b * p.T + t) * p.Hq + kvh * p.G) * D + x % lines * 64));
        }
      }
      // lane i holds page i of a run of 32 pages, and of the next run (its id:
      // of the two next)
      auto load_ids = [&](int q) { return q < npages ? __ldg(trow + q) : 0; };
      auto load_par = [&](int q, int id) {
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (kOneByte) {
          if (q < npages && static_cast<unsigned>(id) < static_cast<unsigned>(p.NB)) {
            const size_t pi = static_cast<size_t>(id) * p.Hkv + kvh;
            if constexpr (kI8) {
              const float2 kp = __ldg(reinterpret_cast<const float2*>(p.k_scale) + pi);
              const float2 vp = __ldg(reinterpret_cast<const float2*>(p.v_scale) + pi);
              r = make_float4(kp.x, kp.y, vp.x, vp.y);
            } else {
              r = make_float4(__ldg(p.k_scale + pi), 0.f, __ldg(p.v_scale + pi), 0.f);
            }
          }
        }
        return r;
      };
      int id = load_ids(lane), id_next = load_ids(lane + 32), id_after = load_ids(lane + 64);
      float4 par = load_par(lane, id), par_next = load_par(lane + 32, id_next);
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++g) {
        const int q0 = j * PPI;  // the step's first page
        if (q0 > 0 && (q0 & 31) == 0) {
          id = id_next;
          par = par_next;
          id_next = id_after;
          par_next = load_par(q0 + 32 + lane, id_next);
          id_after = load_ids(q0 + 64 + lane);
        }
        if (g >= KS && !warp_wait(&k_free[g % KS], ((g - KS) / KS) & 1u)) {
          timed_out = true;
          break;
        }
        volatile TaStep* st = step_at(g);
        const int np = min(PPI, npages - q0);
        const int q = lane - (q0 & 31);  // this lane's page of the step
        const bool mine = q >= 0 && q < np;
        const bool bad = mine && static_cast<unsigned>(id) >= static_cast<unsigned>(p.NB);
        const int phys = bad ? 0 : id;
        auto copy = [&]() {
          uint8_t* dst = sm + L::kK + (g % KS) * L::kKTile;
          uint64_t* bar = kI8 ? &tma_k[g % KS] : &k_full[g % KS];
          if (lane == 0) {
            fence_proxy_async_smem();  // INT8: the converters wrote the stage before
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(np) * (kOneByte ? 128u : 128u * kHalves) * BS);
          }
          __syncwarp();
          if (mine) {
            const int row = p.row_base + (phys * p.Hkv + kvh) * BS;
            if constexpr (kOneByte) {
              tma_load_2d(dst + (kF8K ? 0 : L::kRegion) + q * BS * 128, &kmap, bar, 0, row, policy);
            } else {
#pragma unroll
              for (int h = 0; h < kHalves; ++h) tma_load_2d(dst + h * L::kRegion + q * BS * 128, &kmap, bar, 64 * h, row, policy);
            }
          }
          k_issued = g + 1;
        };
        auto describe = [&]() {
          bool plain = true;
          if constexpr (kOneByte) {
            // vref moves when a step's v scales are more than 2^6 above it, so
            // that P, below 2^8, stays below 2^14 in f16.  (The weights of a
            // page whose scale is below 2^-14 of vref lose bits to f16's
            // subnormals; the mma.sync path has no such limit.)  A scale that is
            // not finite takes no part; P of its page's tokens is NaN, in the
            // rows that attend to them
            const bool finite = fabsf(par.z) < INFINITY;
            const float vm = __uint_as_float(__reduce_max_sync(kFull, mine && finite ? __float_as_uint(fabsf(par.z)) : 0u));
            if (vm > 64.f * vref) vref = vm;
            const float ratio = !mine ? 0.f : !finite ? __uint_as_float(0x7fffffffu) : vref > 0.f ? par.z / vref : 0.f;
            plain = __all_sync(kFull, !mine || (par.x >= 0.f && par.x < INFINITY && par.z > 0.f && par.z < INFINITY));
            if (q >= 0 && q < PPI) {
              const_cast<TaStep*>(step_at(g))->par[q] =
                  make_float4(mine ? par.x : 0.f, kInt8Bias + (mine ? par.y : 0.f), ratio, ratio > 0.f ? __log2f(ratio) : 0.f);
              st->vzero[q] = mine ? par.w : 0.f;
            }
          }
          if (q >= 0 && q < PPI) {
            st->pages[q] = phys;
            st->bad[q] = bad ? 1 : 0;
          }
          if (bad) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
          const int seen = min(t1, base) - (t0 + j * kTreeTokens);  // tokens of the step that every row attends to
          const int flags = (seen < kTreeTokens || __any_sync(kFull, bad) ? kStepMasked : 0) | (plain ? 0 : kStepScales);
          if (lane == 0) {
            st->n = n;
            st->b = b;
            st->kvh = kvh;
            st->t0 = t0;
            st->t1 = t1;
            st->part = part;
            st->np = np;
            st->ctx = ctx;
            st->flags = flags;
            st->vref = vref;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&step_full[g % kTaRing]);  // release: the descriptor
        };
        // one-byte caches: the descriptor takes some 1500 cycles, so the copy
        // first; bf16: the queries wait for the descriptor
        if constexpr (kOneByte) {
          copy();
          describe();
        } else {
          describe();
          copy();
        }
      }
      j0 = 0;
      if (++kvh == p.Hkv) {
        kvh = 0;
        ++b;
      }
    }
    if (!timed_out) {  // no more work
      if (g >= KS && !warp_wait(&k_free[g % KS], ((g - KS) / KS) & 1u)) timed_out = true;
      if (lane == 0 && !timed_out) {
        step_at(g)->n = 0;
        mbar_arrive(&step_full[g % kTaRing]);
      }
    }
  } else if (warp == 18) {
    // V copy warp: V pages of each step
    const uint64_t policy = p.NP > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    for (uint32_t g = 0;; ++g) {
      if (!wait_step(g)) {
        timed_out = true;
        break;
      }
      const volatile TaStep* st = step_at(g);
      if (st->n == 0) break;
      const int kvh = st->kvh, np = st->np;
      if (g >= VS && !warp_wait(&v_free[g % VS], ((g - VS) / VS) & 1u)) {
        timed_out = true;
        break;
      }
      uint8_t* dst = sm + L::kV + (g % VS) * L::kTile;
      uint64_t* bar = kOneByte ? &tma_v[g % VS] : &v_full[g % VS];
      if (lane == 0) {
        fence_proxy_async_smem();  // after the clearing of stale rows and the converters' writes
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(np) * (kOneByte ? 128u : 128u * kHalves) * BS);
      }
      __syncwarp();
      if (lane < np) {
        const int row = p.row_base + (st->pages[lane] * p.Hkv + kvh) * BS;
        if constexpr (kOneByte) {
          tma_load_2d(dst + L::kRegion + lane * BS * 128, &vmap, bar, 0, row, policy);
        } else {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) tma_load_2d(dst + h * L::kRegion + lane * BS * 128, &vmap, bar, 64 * h, row, policy);
        }
      }
      v_issued = g + 1;
    }
  } else if (warp == 19) {
    if constexpr (!kOneByte) {
      // query warp (bf16 caches): each unit's query tiles, once the products
      // with the ones before are done
      uint32_t g0 = 0;
      for (;;) {
        // the products first: only then is the next unit's descriptor at most
        // one turn of the ring away (two turns look alike)
        if ((q_loads > 0 && !warp_wait(q_free, (q_loads - 1) & 1u)) || !wait_step(g0)) {
          timed_out = true;
          break;
        }
        const volatile TaStep* st = step_at(g0);
        const int n = st->n, b = st->b, kvh = st->kvh;
        if (n == 0) break;
        if (lane == 0) mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(L::kQTiles * kHalves) * 128u * static_cast<uint32_t>(p.G * p.Tt));
        __syncwarp();
        if (lane < L::kQTiles * kHalves) {  // rows past T are zero-filled
          const int i = lane / kHalves, half = lane % kHalves;
          tma_load_4d(sm + L::kQ + i * L::kTile + half * L::kRegion, &qmap, q_full, 64 * half, kvh * p.G, (2 * pair + i) * p.Tt, b);
        }
        ++q_loads;
        g0 += static_cast<uint32_t>(n);
      }
    }
  } else if (warp == 16) {
    if (elect_one()) {
      constexpr uint32_t kIdescS = kF8K       ? tc_idesc_e4m3_f32(kTaRows, kTreeTokens)
                                   : kOneByte ? tc_idesc_f16_f32(kTaRows, kTreeTokens)
                                              : tc_idesc_bf16_f32(kTaRows, kTreeTokens);
      constexpr uint32_t kIdescO = kOneByte ? tc_idesc_f16_f32(kTaRows, D, /*b_mn_major=*/true)
                                            : tc_idesc_bf16_f32(kTaRows, D, /*b_mn_major=*/true);
      // operand descriptors of stage 0; a later stage or slice adds its byte
      // offset / 16 to the start-address field
      const uint64_t q_desc = tc_smem_desc(smem_addr(sm + L::kQ), 16, 1024, 2);
      const uint64_t k_desc = tc_smem_desc(smem_addr(sm + L::kK), 16, 1024, 2);
      const uint64_t v_desc = tc_smem_desc(smem_addr(sm + L::kV), L::kRegion, 1024, 2);
      // S_i = Q . K^T; A and B K-major with the 128-byte swizzle, 32 bytes of
      // each row per product.  (Loops of two products: the issuing thread's
      // code is fetched anew each step, between the softmax warps'.)
      auto issue_s = [&](int i, uint32_t stage) {
        const uint64_t qd = q_desc + (PAIR ? i * (L::kTile >> 4) : 0u), kd = k_desc + stage * (L::kKTile >> 4);
        constexpr int kParts = kF8K ? 2 : kHalves;  // regions of the query: E4M3 both parts against the same codes
#pragma unroll 1
        for (int h = 0; h < kParts; ++h) {
          const uint64_t qh = qd + h * (L::kRegion >> 4), kh = kd + (kF8K ? 0u : h * (L::kRegion >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (kF8K)
              tc_mma_e4m3(tmem + 128u * i, qh + 2 * kk, kh + 2 * kk, kIdescS, h > 0 || kk > 0);
            else
              tc_mma_bf16(tmem + 128u * i, qh + 2 * kk, kh + 2 * kk, kIdescS, h > 0 || kk > 0);
          }
        }
        ++mma_issued;
      };
      // O_i (+)= P_i . V: P of a half's tokens 16kk .. 16kk + 15 in columns
      // 8kk .. +7 of the half's 64 columns of S_i, V MN-major as the pages hold
      // it (64-d halves kRegion apart, 8-token groups 1024 B apart)
      uint32_t pc[2] = {0, 0};  // P tiles taken, per stream
      uint32_t ks = 0, kph = 0, vs = 0, vph = 0;  // stage and phase of the next K and V
      auto issue_pv = [&](int i, bool first, uint32_t iu) -> bool {
        if (!ta_wait(&p_full[i], pc[i] & 1u)) return false;
        ++pc[i];
        if ((!PAIR || i == 0) && !ta_wait(&v_full[vs], vph)) return false;
        if (first && iu > 0 && !ta_wait(&o_free[i], (iu - 1) & 1u)) return false;
        tc_fence_after_sync();
        const uint64_t vd = v_desc + vs * (L::kTile >> 4);
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_bf16_ts(tmem + 256u + 128u * i, tmem + 128u * i + 64u * h + 8u * kk, vd + (h * 4 + kk) * (2048 >> 4), kIdescO,
                           !first || h > 0 || kk > 0);
        ++mma_issued;
        if (!PAIR || i == 1) {
          tc_commit(&v_free[vs]);
          if (++vs == VS) {
            vs = 0;
            vph ^= 1u;
          }
        }
        return true;
      };
      uint32_t g0 = 0;
      bool ok = true;
      for (uint32_t iu = 0;; ++iu) {
        if (!(ok = ta_wait(&step_full[g0 % kTaRing], (g0 / kTaRing) & 1u))) break;
        const int n = step_at(g0)->n;
        if (n == 0) break;
        if (!(ok = ta_wait(q_full, iu & 1u))) break;
        const int events = PAIR ? 2 * n : n;
#pragma unroll 1
        for (int e = 0; ok && e < events; ++e) {
          const int i = e & 1, k = e >> 1;  // stream, its step
          if (k > 0 && !(ok = issue_pv(i, k == 1, iu))) break;
          if ((!PAIR || i == 0) && !(ok = ta_wait(&k_full[ks], kph))) break;
          tc_fence_after_sync();
          issue_s(i, ks);
          tc_commit(&s_full[i]);
          if (!PAIR || i == 1) {
            tc_commit(&k_free[ks]);
            if (++ks == KS) {
              ks = 0;
              kph ^= 1u;
            }
          }
          if (e == events - 1) tc_commit(q_free);
        }
        // the last products of both streams, the earlier step's first
#pragma unroll 1
        for (int x = 0; ok && x < 2; ++x) {
          const int i = (!PAIR && (n & 1)) ? 1 - x : x;
          const int ni = PAIR ? n : (n + 1 - i) / 2;  // the stream's steps
          if (ni == 0) continue;
          if (!(ok = issue_pv(i, ni == 1, iu))) break;
          tc_commit(&o_full[i]);
        }
        if (!ok) break;
        g0 += static_cast<uint32_t>(n);
      }
      if (!ok) timed_out = true;
    }
    __syncwarp();
  }
  } else if (warp >= 20) {
    if constexpr (kOneByte) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ta_role_regs(KV)));
      // converter warps: 16 rows each of a unit's query tiles, then of its
      // steps' V and INT8 K
      const int cw = warp - 20;
      constexpr int kRows = kTreeTokens / kConvWarps;
      static_assert(kRows == 16, "");
      auto convert = [&](bool is_k, uint32_t g) {
        const int row0 = kRows * cw;
        uint8_t* st = (is_k ? sm + L::kK + (g % KS) * L::kKTile : sm + L::kV + (g % VS) * L::kTile) + row0 * 128;
        const volatile TaStep* sp = step_at(g);
        const int rows = sp->np * BS - row0;  // of the step's pages
        if (is_k) {
          widen_rows<KV, kI8>(st, L::kRegion, lane, 0u, rows);
        } else {
          uint32_t zc = 0u;
          if constexpr (kI8) {
            if ((lane & 15) < rows) zc = int8_zero_const(sp->vzero[row0 / BS]);
          }
          widen_rows<KV, false>(st, L::kRegion, lane, zc, rows);
        }
        fence_proxy_async_smem();  // read by the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(is_k ? &k_full[g % KS] : &v_full[g % VS]);
      };
      uint32_t g0 = 0;
      for (uint32_t iu = 0;; ++iu) {
        if (!wait_step(g0)) {
          timed_out = true;
          break;
        }
        const int n = step_at(g0)->n, b = step_at(g0)->b, kvh = step_at(g0)->kvh;
        if (n == 0) break;
        // the query tiles of the unit before are done with, and every softmax
        // warp has seen its q_full: a stream without a step in that unit would
        // otherwise be overtaken by this unit's (two phases look alike)
        if (iu > 0 && !(warp_wait(q_free, (iu - 1) & 1u) && warp_wait(q_read, (iu - 1) & 1u))) {
          timed_out = true;
          break;
        }
        // Query row scaled by 2^-kq, in the type of the K operand.  INT8: f16,
        // largest |q| in [2^14, 2^15), exact within 2^-10 of it.  E4M3: largest
        // |q'| in [2^7, 2^8) as qh = e4m3(q') and ql = e4m3(q' - qh): a bf16
        // q' has 8 significant bits, 4 in each part, so the sum is exact from
        // 2^-2 up and within 2^-10 below
        // Two lanes a row: 64 elements each, to 16 bits (f16 holds every q'
        // above 2^-14 exactly) and from there to the two parts.
        float2* qrow = reinterpret_cast<float2*>(sm + L::kQrow);
        const int r = kRows * cw + (lane & 15), half = lane >> 4;
#pragma unroll 1
        for (int i = 0; i < L::kQTiles; ++i) {
          const int tl = r / p.G, t = (2 * pair + i) * p.Tt + tl;
          const bool in = tl < p.Tt && t < p.T;
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (static_cast<size_t>(b * p.T + (in ? t : 0)) * p.Hq + kvh * p.G + (in ? r - tl * p.G : 0)) * D + 64 * half);
          uint32_t mx = 0;  // largest |q| as bf16 bits, of both 16-bit halves
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 w = __ldg(src + c);
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
          }
          mx = max(mx & 0xffffu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(kFull, mx, 16));
          if (!in) mx = 0;
          const int kq = mx == 0 ? 0 : max(-100, min(100, static_cast<int>(mx >> 7) - 127 - (kF8K ? 7 : 14)));
          const float sc = __uint_as_float(static_cast<uint32_t>(127 - kq) << 23);  // 2^-kq
          float qsum = 0.f;
          uint8_t* qt = sm + L::kQ + i * L::kTile + r * 128 + (kF8K ? 0u : half * L::kRegion);
#pragma unroll 1
          for (int c2 = 0; c2 < 4; ++c2) {  // 16 elements
            uint32_t wf[8], wl[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 w = __ldg(src + 2 * c2 + h);
              const uint32_t w4[4] = {in ? w.x : 0u, in ? w.y : 0u, in ? w.z : 0u, in ? w.w : 0u};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t f = pack_f16x2(bf16lo_to_f32(w4[e]) * sc, bf16hi_to_f32(w4[e]) * sc);
                if constexpr (kF8K) {
                  const __half2_raw fr = *reinterpret_cast<const __half2_raw*>(&f);
                  const __nv_fp8x2_storage_t hi = __nv_cvt_halfraw2_to_fp8x2(fr, __NV_SATFINITE, __NV_E4M3);
                  const __half2 rest = __hsub2(__half2(fr), __half2(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3)));
                  const __nv_fp8x2_storage_t lo = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(rest), __NV_SATFINITE, __NV_E4M3);
                  const int k = 2 * h + (e >> 1), s = 16 * (e & 1);
                  wf[k] = (s ? wf[k] : 0u) | static_cast<uint32_t>(hi) << s;
                  wl[k] = (s ? wl[k] : 0u) | static_cast<uint32_t>(lo) << s;
                } else {
                  wf[4 * h + e] = f;
                  const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&f));
                  qsum += fv.x + fv.y;
                }
              }
            }
            const int c = kF8K ? 4 * half + c2 : 2 * c2;
            *reinterpret_cast<uint4*>(qt + ((c ^ (r & 7)) << 4)) = make_uint4(wf[0], wf[1], wf[2], wf[3]);
            if constexpr (kF8K)
              *reinterpret_cast<uint4*>(qt + L::kRegion + ((c ^ (r & 7)) << 4)) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
            else
              *reinterpret_cast<uint4*>(qt + (((c + 1) ^ (r & 7)) << 4)) = make_uint4(wf[4], wf[5], wf[6], wf[7]);
          }
          qsum += __shfl_xor_sync(kFull, qsum, 16);
          // (a row with an infinity or NaN is NaN, as E4M3 codes cannot hold it)
          const float back = mx < 0x7f80u ? __uint_as_float(static_cast<uint32_t>(127 + kq) << 23) : __uint_as_float(0x7fffffffu);
          if (half == 0) qrow[i * kTaRows + r] = make_float2(back, qsum);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        // Each warp takes what has landed: K of a step before V of the step
        // before it, the order that the products need them in, but whichever
        // is there first (in that order alone: INT8 1.72 instead of 1.65 us a
        // step, 2.8 or more instead of 2.67 for two tiles).
        auto there = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_test_wait(bar, parity)) != 0; };
        int jk = kI8 ? 0 : n, jv = 0, tries = 0;  // next K and V of the unit
        while (jk < n || jv < n) {
          const uint32_t gk = g0 + jk, gv = g0 + jv;
          auto k_there = [&]() { return jk < n && there(&step_full[gk % kTaRing], (gk / kTaRing) & 1u) && there(&tma_k[gk % KS], (gk / KS) & 1u); };
          auto v_there = [&]() { return jv < n && there(&step_full[gv % kTaRing], (gv / kTaRing) & 1u) && there(&tma_v[gv % VS], (gv / VS) & 1u); };
          const bool k_first = kI8 && jk <= jv + 1;
          const bool take_k = kI8 && ((k_first && k_there()) || (!k_first && !v_there() && k_there()));
          if (take_k) {
            convert(true, gk);
            ++jk;
            tries = 0;
          } else if (v_there()) {
            convert(false, gv);
            ++jv;
            tries = 0;
          } else {
            if (++tries > kConvTries) break;
            __nanosleep(20);
          }
        }
        const bool ok = jk == n && jv == n;
        if (!ok) {
          timed_out = true;
          break;
        }
        g0 += static_cast<uint32_t>(n);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(ta_soft_regs(KV)));
    // softmax warps: stream i, row r of its tile in TMEM lane r, half hh of
    // the step's tokens.  Two warps share 32 rows: both hold the same running
    // maximum of a row, and each the sum of its own half.
    const int i = warp >> 3, hh = (warp >> 2) & 1, r = 32 * (warp & 3) + lane;
    const int pair_bar = 1 + (warp & 3) + 4 * i;  // named barrier of the two warps
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + 128u * i;
    const uint32_t t_o = tmem + lane_base + 256u;  // O0; O1 is 128 columns on
    const float c = p.scale_log2;
    const int tile = PAIR ? 2 * pair + i : 0;
    const int tl = r / p.G, t = tile * p.Tt + tl;
    const bool in_tile = tl < p.Tt && t < p.T;
    // warps without rows only keep the barriers' counts and clear stale V rows
    const bool warp_dead = !__any_sync(kFull, in_tile);
    float* xch = reinterpret_cast<float*>(sm + L::kXml);
    float* x_mine = xch + (2 * i + hh) * kTaRows + r;
    const float* x_other = xch + (2 * i + (hh ^ 1)) * kTaRows + r;
    uint32_t g0 = 0, steps = 0, units1 = 0;  // steps of this stream, units with a step for stream 1
    // A wait of this warp gave up: it waits for nothing more, and leaves with
    // the warp that shares its rows, at their next barrier
    bool fail = false, left = false;
    for (uint32_t iu = 0;; ++iu) {
      if (!wait_step(g0)) fail = true;
      if (bar_red_or(pair_bar, 64, fail)) {
        fail = true;
        break;
      }
      int n, b, kvh, t0, t1, part, base, mrow, prow, row_state;
      {
        const volatile TaStep* st = step_at(g0);
        n = st->n;
        if (n == 0) break;
        b = st->b;
        kvh = st->kvh;
        t0 = st->t0;
        t1 = st->t1;
        part = st->part;
        const int nodes = p.tree.node_counts != nullptr ? __ldg(p.tree.node_counts + b) : p.T;
        base = st->ctx - nodes;
        const bool live = in_tile && t < nodes;
        mrow = live ? b * p.tree.stride + t * p.tree.words : -1;
        prow = (b * p.Hkv + kvh) * p.tree.words;
        row_state = live ? kTreeRowNormal : kTreeRowZero;
      }
      float cq = c, qsum = 0.f, vref = 1.f;
      if constexpr (kOneByte) {
        if (!fail && !warp_wait(q_full, iu & 1u)) fail = true;
        const float2 qr = reinterpret_cast<const float2*>(sm + L::kQrow)[(PAIR ? i * kTaRows : 0) + r];
        cq = c * qr.x;
        qsum = qr.y;
        __syncwarp();
        if (lane == 0) mbar_arrive(q_read);
      }
      float m = -INFINITY, l = 0.f;  // log2-domain lazy running maximum of the row, sum of this half
      const int ni = PAIR ? n : (n + 1 - i) / 2;  // this stream's steps
#pragma unroll 1
      for (int k = 0; k < ni; ++k, ++steps) {
        const int j = PAIR ? k : 2 * k + i;
        const uint32_t g = g0 + j;
        const int pos0 = t0 + j * kTreeTokens;
        const int nvs = t1 - pos0;  // tokens of the step in the sequence
        if (!fail && !ta_wait(&step_full[g % kTaRing], (g / kTaRing) & 1u)) fail = true;
        const TaStep* st = const_cast<const TaStep*>(step_at(g));
        const int flags = *reinterpret_cast<const volatile int*>(&st->flags);
        uint64_t badw = 0ull, bad0 = 0ull, bad1 = 0ull;  // bad pages; nodes with a non-finite V row
        uint64_t rm = ~0ull;                             // this half's tokens that the row attends to
        // (rows past the sequence's nodes attend to every token before them
        // too: their output is zero whatever they attend to)
        if (flags & kStepMasked) {
          badw = PPI == 8 ? *reinterpret_cast<const volatile uint64_t*>(st->bad) : *reinterpret_cast<const volatile uint32_t*>(st->bad);
          const bool nodes_here = pos0 + kTreeTokens > base;
          if (nodes_here && p.tree.poison != nullptr) {
            bad0 = tree_window64(p.tree.poison + prow, p.tree.words, pos0 - base);
            bad1 = tree_window64(p.tree.poison + prow, p.tree.words, pos0 - base + 64);
          }
          rm = low_bits64(nvs - 64 * hh);
#pragma unroll
          for (int q = 0; q < PPI / 2; ++q)
            if ((badw >> (8 * (q + hh * (PPI / 2)))) & 0xffu) rm &= ~(((1ull << BS) - 1ull) << (q * BS));
          uint64_t see = low_bits64(base - pos0 - 64 * hh);
          if (nodes_here && mrow >= 0) see |= tree_window64(p.tree.mask + mrow, p.tree.words, pos0 - base + 64 * hh);
          rm &= see;
          const uint64_t badh = hh ? bad1 : bad0;
          if ((rm & badh) && row_state == kTreeRowNormal) row_state = kTreeRowNan;
          rm &= ~badh;
        }
        bool vgrow = false;
        float factor = 1.f;
        if constexpr (kOneByte) {
          const float vnew = *reinterpret_cast<const volatile float*>(&st->vref);
          if (vnew != vref) {  // (0 until a page has a scale: O is 0 so far)
            if (k > 0 && vref != 0.f) {
              factor = vref / vnew;
              vgrow = true;
            }
            vref = vnew;
          }
        }
        const bool plain = flags == 0 && c >= 0.f;  // (a lower scale turns the order of the scores)
        if (!fail && !ta_wait(&s_full[i], steps & 1u)) fail = true;
        __syncwarp();
        tc_fence_after_sync();
        if (!warp_dead) {
          const uint32_t t_h = t_s + 64u * hh;  // this half's scores, then its P over them
          if (!plain) {
            // Scores to log2 units, -inf where masked, back to where they
            // came from.  Once or twice an item, so a short loop: code that
            // runs rarely costs its fetch, some 20 cycles an instruction.
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t y[16];
              tc_ld16(t_h + 16u * q, y);
              tc_wait_ld_regs16(y);
              float ck = c, add = 0.f;
              if constexpr (kOneByte) {
                const float4 pr = st->par[(64 * hh + 16 * q) / BS];
                ck = cq * pr.x;
                if constexpr (kI8) add = -pr.y * qsum * ck;
              }
              const uint32_t mk = static_cast<uint32_t>(rm >> (16 * q));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  z[e] = __float_as_uint(((mk >> (8 * h + e)) & 1u) ? fmaf(__uint_as_float(y[8 * h + e]), ck, add) : -INFINITY);
                tc_st8(t_h + 16u * q + 8u * h, z);
              }
            }
            tc_wait_st();
          }
          uint32_t x0[32], x1[32];
          tc_ld32(t_h, x0);
          tc_ld32(t_h + 32u, x1);
          tc_wait_ld_regs(x0);
          tc_regs_loaded(x1);
          // coefficients of the scores of page h of the half's 32 tokens c32:
          // a score in log2 units is x ck + add, P x v scale / vref is
          // 2^(score - m + lv)
          auto page = [&](int c32, int h, float& ck, float& add, float& lv) {
            const float4 pr = st->par[(64 * hh + 32 * c32) / BS + h];
            ck = plain ? cq * pr.x : 1.f;
            add = kI8 && plain ? -pr.y * qsum * ck : 0.f;  // the biased K codes
            lv = pr.w;
          };
          const float c_u = plain ? c : 1.f;
          auto ext32 = [&](const uint32_t (&x)[32], int c32) -> float {  // largest score, in log2 units
            if constexpr (!kOneByte) {
              return tree_ext32<true>(x) * c_u;
            } else if constexpr (BS == 32) {
              float ck, add, lv;
              page(c32, 0, ck, add, lv);
              return fmaf(tree_ext32<true>(x), ck, add);
            } else {
              float ck, add, lv;
              page(c32, 0, ck, add, lv);
              const float e0 = fmaf(max16(x, 0), ck, add);
              page(c32, 1, ck, add, lv);
              return fmaxf(e0, fmaf(max16(x, 16), ck, add));
            }
          };
          float smax = fmaxf(ext32(x0, 0), ext32(x1, 1));
          // lazy maximum: moved when the row's exceeds it by more than 2^8
          const bool want = m == -INFINITY ? smax != -INFINITY : smax > m + 8.f;
          bool grow = false;
          if (bar_red_or(pair_bar, 64, want || fail)) {
            *x_mine = smax;
            if (bar_red_or(pair_bar, 64, fail)) {
              fail = left = true;
              break;
            }
            smax = fmaxf(smax, *x_other);
            grow = m == -INFINITY ? smax != -INFINITY : smax > m + 8.f;
            if (grow) {
              const float f = (m == -INFINITY) ? 0.f : ex2_approx(m - smax);
              factor *= f;
              l *= f;
              m = smax;
            }
            __syncwarp();
          }
          const float neg_m = (m == -INFINITY) ? 0.f : -m;
          float ps0 = 0.f, ps1 = 0.f;
          auto write_p = [&](const uint32_t (&x)[32], int c32) {
            float ck = c_u, add = 0.f, lv = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16 scores
              if constexpr (kOneByte) {
                if (h == 0 || BS == 16) {
                  page(c32, h, ck, add, lv);
                  ps0 = ps1 = 0.f;
                }
              }
              uint32_t pw[8];
              const float bias = add + neg_m + lv;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int k2 = 16 * h + 2 * e;
                float a0, a1;
                ffma2(a0, a1, __uint_as_float(x[k2]), __uint_as_float(x[k2 + 1]), ck, ck, bias, bias);
                const float p0 = ex2_approx(a0);
                const float p1 = ex2_approx(a1);
                fadd2(ps0, ps1, ps0, ps1, p0, p1);
                pw[e] = kOneByte ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
              }
              if constexpr (kOneByte) {
                if (h == 1 || BS == 16) l = fmaf(ps0 + ps1, ex2_approx(-lv), l);
              }
              tc_st8(t_h + 16 * c32 + 8 * h, pw);
            }
          };
          if (!kOneByte || !(flags & kStepScales)) {
            if constexpr (kOneByte) {
              // one-byte caches: the second 32 scores are read again, so that
              // 32 registers less are held meanwhile (the first 32's P covers
              // only columns that are done with)
              write_p(x0, 0);
              tc_ld32(t_h + 32u, x1);
              tc_wait_ld_regs(x1);
              write_p(x1, 1);
            } else {
              write_p(x0, 0);
              write_p(x1, 1);
              l += ps0 + ps1;
            }
          } else {
            // a page's v scale is zero, negative or not finite
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t y[16], pw[8];
              tc_ld16(t_h + 16u * q, y);
              tc_wait_ld_regs16(y);
              const float vr = st->par[(64 * hh + 16 * q) / BS].z;
              const uint32_t mk = static_cast<uint32_t>(rm >> (16 * q));
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float p0 = ex2_approx(__uint_as_float(y[2 * e]) + neg_m);
                const float p1 = ex2_approx(__uint_as_float(y[2 * e + 1]) + neg_m);
                l += p0 + p1;
                // (a masked token's page may have no finite scale: 0 x that would be NaN)
                pw[e] = pack_f16x2(((mk >> (2 * e)) & 1u) ? p0 * vr : 0.f, ((mk >> (2 * e + 1)) & 1u) ? p1 * vr : 0.f);
              }
              tc_st8(t_h + 8u * q, pw);
            }
          }
          // O_i of the steps before, rarely, half of the columns by each warp
          // (quiescent: PV_i of the step before was done before this S_i, the
          // next waits for p_full)
          if (k > 0 && __any_sync(kFull, grow || vgrow)) {
#pragma unroll 1
            for (int oc = hh * (D / 2); oc < (hh + 1) * (D / 2); oc += 32) {
              uint32_t ov[32];
              tc_ld32(t_o + 128u * i + oc, ov);
              tc_wait_ld_regs(ov);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float a, b2;
                fmul2(a, b2, __uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), factor, factor);
                ov[e] = __float_as_uint(a);
                ov[e + 1] = __float_as_uint(b2);
              }
              tc_st32(t_o + 128u * i + oc, ov);
            }
          }
        }
        // V rows of tokens outside the sequence or of a bad page may hold
        // anything, and nodes' V rows that are not finite would reach every
        // row, while P is 0 there: once V has landed, the threads of row r
        // clear it (a pair's streams write the same zeros)
        if ((flags & kStepMasked) && (nvs < kTreeTokens || badw != 0 || (bad0 | bad1) != 0ull)) {
          if (!fail && !warp_wait(&v_full[g % VS], (g / VS) & 1u)) fail = true;
          if (fail) {
          } else if (r >= nvs || ((badw >> (8 * (r / BS))) & 0xffu) || (((r < 64 ? bad0 : bad1) >> (r & 63)) & 1ull)) {
            // 64-d half hh (head_dim 64: 32 d)
            uint8_t* vb = sm + L::kV + (g % VS) * L::kTile + r * 128 + (kHalves == 2 ? hh * L::kRegion : hh * 64);
#pragma unroll
            for (int cc = 0; cc < 4 * kHalves; ++cc) *reinterpret_cast<uint4*>(vb + 16 * cc) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();  // read by the tensor cores
          __syncwarp();
        }
        tc_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i]);
      }
      if (left) break;

      // the unit's output: O / l as bf16, or a partial (m, l, O)
      // a row that attends to a node with a non-finite V row is NaN in every
      // column, also those that other warps write: through its sum
      if (row_state == kTreeRowNan) l = tree_row_value(kTreeRowNan);
      if (row_state == kTreeRowZero) {  // whatever its query held
        m = -INFINITY;
        l = 0.f;
      }
      float f0 = kOneByte ? vref : 1.f, f1 = 0.f;
      if constexpr (PAIR) {
        if (!fail && !warp_wait(&o_full[i], iu & 1u)) fail = true;
        *x_mine = l;
        if (bar_red_or(pair_bar, 64, fail)) {
          fail = true;
          break;
        }
        l += *x_other;
      } else {
        // both streams' last products; their completion also means that what
        // was exchanged for the unit before has been read
        if (!fail && !warp_wait(&o_full[0], iu & 1u)) fail = true;
        if (n > 1) {
          if (!fail && !warp_wait(&o_full[1], units1 & 1u)) fail = true;
          ++units1;
        }
        float* xl = xch + 4 * kTaRows;  // [stream][half][128]
        float* xm = xl + 4 * kTaRows;   // [stream][128]
        float* xv = xm + 2 * kTaRows;   // [stream]
        xl[(2 * i + hh) * kTaRows + r] = l;
        if (hh == 0) xm[i * kTaRows + r] = m;
        if (kOneByte && hh == 0 && r == 0) xv[i] = vref;
        __syncwarp();
        if (lane == 0) mbar_arrive(x_full);
        if (!fail && !warp_wait(x_full, iu & 1u)) fail = true;
        if (bar_red_or(pair_bar, 64, fail)) {
          fail = true;
          break;
        }
        const float m0 = xm[r], m1 = xm[kTaRows + r];
        const float l0 = xl[r] + xl[kTaRows + r], l1 = xl[2 * kTaRows + r] + xl[3 * kTaRows + r];
        m = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - m);
        f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
        l = f0 * l0 + f1 * l1;
        if constexpr (kOneByte) {  // O_i is in units of its stream's vref
          f0 *= xv[0];
          f1 *= xv[1];
        }
      }
      tc_fence_after_sync();
      if (!warp_dead) {
        const int h = kvh * p.G + (r - tl * p.G);
        const size_t qrow = static_cast<size_t>(b * p.T + t) * p.Hq + h;
        const size_t prow_o = (static_cast<size_t>(blockIdx.x) * 2 + (part - 1)) * (L::kQTiles * kTaRows) + (PAIR ? i * kTaRows : 0) + r;
        if (part == 0) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          f0 *= inv;
          f1 *= inv;
        }
        // a pair's warp: half of its tile's columns; else a quarter of the one tile's
        constexpr int kCols = PAIR ? D / 2 : D / 4;
        const int c0 = (PAIR ? hh : 2 * i + hh) * kCols;
#pragma unroll 1
        for (int cc = c0; cc < c0 + kCols; cc += 16) {
          uint32_t ov[16], o1[16];
          tc_ld16(t_o + (PAIR ? 128u * i : 0u) + cc, ov);
          if constexpr (!PAIR) {  // (O1 of a unit with one step holds anything)
            tc_ld16(t_o + 128u + cc, o1);
          }
          tc_wait_ld_regs16(ov);
          if constexpr (!PAIR) tc_regs_loaded16(o1);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float a, b2;
            fmul2(a, b2, __uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), f0, f0);
            if constexpr (!PAIR) {
              const float z0 = n > 1 ? __uint_as_float(o1[e]) : 0.f, z1 = n > 1 ? __uint_as_float(o1[e + 1]) : 0.f;
              a = fmaf(z0, f1, a);
              b2 = fmaf(z1, f1, b2);
            }
            ov[e] = row_state == kTreeRowZero ? 0u : __float_as_uint(a);
            ov[e + 1] = row_state == kTreeRowZero ? 0u : __float_as_uint(b2);
          }
          if (in_tile) {
            if (part == 0) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + qrow * D + cc);
#pragma unroll
              for (int c8 = 0; c8 < 2; ++c8) {
                const float* f = reinterpret_cast<const float*>(ov + 8 * c8);
                dst[c8] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow_o * D + cc);
#pragma unroll
              for (int c4 = 0; c4 < 4; ++c4) dst[c4] = make_uint4(ov[4 * c4], ov[4 * c4 + 1], ov[4 * c4 + 2], ov[4 * c4 + 3]);
            }
          }
          __syncwarp();  // the next TMEM load is warp-collective
        }
        if (in_tile && part != 0 && hh == 0 && (PAIR || i == 0)) p.part_ml[prow_o] = make_float2(m, l);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&o_free[i]);
        if (!PAIR) mbar_arrive(&o_free[1 - i]);
      }
      g0 += static_cast<uint32_t>(n);
    }
    if (fail) timed_out = true;
  }

  timed_out = __syncthreads_or(timed_out) != 0;  // every role has left its loop
  if (timed_out) {
    if (tid == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    // each role lets its own copies and products still in flight finish
    // (bounded) before the shared and tensor memory are released
    if (warp == 17 && lane == 0)
#pragma unroll 1
      for (uint32_t g = k_issued > KS ? k_issued - KS : 0; g < k_issued; ++g)
        mbar_wait_bounded(kI8 ? &tma_k[g % KS] : &k_full[g % KS], (g / KS) & 1u, kWaitLimitNs / 16);
    if (warp == 18 && lane == 0) {
#pragma unroll 1
      for (uint32_t g = v_issued > VS ? v_issued - VS : 0; g < v_issued; ++g)
        mbar_wait_bounded(kOneByte ? &tma_v[g % VS] : &v_full[g % VS], (g / VS) & 1u, kWaitLimitNs / 16);
    }
    if (warp == 19 && lane == 0 && q_loads > 0) mbar_wait_bounded(q_full, (q_loads - 1) & 1u, kWaitLimitNs / 16);
    if (warp == 16 && mma_issued > 0) {  // one commit covers every product issued
      tc_commit(mma_drain);
      mbar_wait_bounded(mma_drain, 0, kWaitLimitNs / 16);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) tc_dealloc(tmem, kTaCols);
}

}  // namespace pkv
