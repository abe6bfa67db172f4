// Merge of the partials that the tcgen05 attention of drafted trees and of
// packed rows leaves.
#pragma once

#include <type_traits>

#include "tree_attend.cuh"

namespace pkv {

// out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p over the partials
// of an item that shares split.  The share in which the item starts leaves it
// as its last unit; the shares after it continue it with their first unit
// until one ends it.
//
// One CTA per (share, row tiles of a CTA, 16 or 32 rows), a warp per two or four
// rows.  The partials are in L2 and few, so it is a chain of loads: bounds, a
// lane each (packed rows: one record of the share), then m and l of the parts of
// all rows by one load of the warp, next to the rows of the first parts.  (A
// warp per row in turn, with the loads after the maxima, took 5 us longer for
// 151 split items of 128 rows.)  Four rows a warp for the packed rows' pairs of
// tiles, where items are long and have two or three parts: 151 items of 256 rows
// 11 us instead of 16 after a cold start; two elsewhere, where a short item may
// have many (one request of five rows: 15.8 us a call instead of 17.6).
constexpr int kTreeMergeThreads = 256;
__host__ __device__ constexpr int merge_cta_rows(int rows) { return kTreeMergeThreads / 32 * rows; }  // of a CTA

struct TreeMergeArgs {
  const TreeBound* bounds;
  const PackedMerge* merge;  // packed rows
  const int32_t* shares;
  const float2* part_ml;
  const float* part_o;
  __nv_bfloat16* out;
  int Hq, G, T, Tt, NP, tiles /* per CTA */;
};

template <int D, bool PACKED, int ROWS>  // rows of a warp
__global__ void __launch_bounds__(kTreeMergeThreads, 3) tree_merge_kernel(const TreeMergeArgs a) {
  constexpr int kPer = D / 32, kRows = ROWS, kLanes = 32 / kRows, kBatch = 8 / ROWS;  // (parts at a time)
  pdl_trigger();
  pdl_wait();
  const int rows = a.tiles * kTaRows, slices = rows / merge_cta_rows(ROWS);
  const int slice = blockIdx.x % slices;
  const int cta = blockIdx.x / slices;
  const int share = cta / a.NP, pair = cta - share * a.NP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int parts, place, kvh, first_row, tokens;  // the rows of q that tile 0 starts with, and how many there are
  if constexpr (PACKED) {
    const int4 d = __ldg(reinterpret_cast<const int4*>(a.merge + share));
    kvh = __ldg(&a.merge[share].kvh);
    if (d.x == 0) return;
    parts = d.x;
    place = d.y;
    first_row = d.z;
    tokens = d.w;
  } else {
    // (the grid leaves out the last share that the workspace has room for)
    const int shares = *a.shares;
    const TreeBound mine = a.bounds[share], next = a.bounds[share + 1];
    if (!tree_splits(mine, next, share, shares)) return;
    place = tree_split_place(mine, next);
    int last = share + 1;  // the share that ends the item
#pragma unroll 1
    for (;;) {
      const int s = last + 1 + lane;
      bool ends = true;
      if (s < shares) ends = tree_item_ends(next, a.bounds[s]);
      const unsigned found = __ballot_sync(kFull, ends);
      last += found ? __ffs(found) - 1 : 32;
      if (found) break;
    }
    parts = last - share + 1;
    kvh = next.kvh;
    first_row = next.b * a.T;
    tokens = a.T;
  }
  const size_t first = (static_cast<size_t>(cta) * 2 + place) * rows;
  const size_t stride = static_cast<size_t>(a.NP) * 2 * rows;  // from a share's partials to the next one's
  const size_t cont = (static_cast<size_t>(cta) * 2) * rows;
  const int rr0 = slice * merge_cta_rows(ROWS) + warp * kRows;
  const int tile = (a.tiles == 2 ? 2 * pair : 0) + rr0 / kTaRows;
  unsigned live = 0;  // rows with a node
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int tl = (rr0 + k) % kTaRows / a.G;
    if (tl < a.Tt && tile * a.Tt + tl < tokens) live |= 1u << k;
  }
  if (live == 0) return;
  auto at = [&](int k, int p) { return (p == 0 ? first : cont + stride * p) + rr0 + k; };
  using Vec = std::conditional_t<kPer == 4, float4, float2>;
  auto load = [&](int k, int p) -> Vec {
    Vec v{};
    if (p < parts && ((live >> k) & 1u)) v = *reinterpret_cast<const Vec*>(a.part_o + at(k, p) * D + lane * kPer);
    return v;
  };
  Vec v[kBatch][kRows];  // parts at a time
#pragma unroll
  for (int q = 0; q < kBatch; ++q)
#pragma unroll
    for (int k = 0; k < kRows; ++k) v[q][k] = load(k, q);
  const int mk = lane / kLanes, mp = lane % kLanes;  // this lane's row and part
  auto load_ml = [&](int p) { return p < parts && ((live >> mk) & 1u) ? a.part_ml[at(mk, p)] : make_float2(-INFINITY, 0.f); };
  float2 ml = load_ml(mp);
  float M = ml.x;
#pragma unroll 1
  for (int p = mp + kLanes; p < parts; p += kLanes) M = fmaxf(M, load_ml(p).x);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  float acc[kRows][kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kRows; ++k)
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc[k][j] = 0.f;
#pragma unroll 1
  for (int p0 = 0; p0 < parts; p0 += kLanes) {
    if (p0 > 0) ml = load_ml(p0 + mp);
    // (an empty partial has O = 0, or the row's fixed value)
    const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
    sum = fmaf(w, ml.y, sum);
    const int pn = min(kLanes, parts - p0);
#pragma unroll 1
    for (int pp = 0; pp < pn; pp += kBatch) {
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          const float wq = __shfl_sync(kFull, w, kLanes * k + pp + q);  // (0 past the last part, and its row zeros)
          const float* x = reinterpret_cast<const float*>(&v[q][k]);
#pragma unroll
          for (int j = 0; j < kPer; ++j) acc[k][j] = fmaf(wq, x[j], acc[k][j]);
          v[q][k] = load(k, p0 + pp + kBatch + q);
        }
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  const float inv_mine = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const float inv = __shfl_sync(kFull, inv_mine, kLanes * k);
    if (!((live >> k) & 1u)) continue;
    const int r = (rr0 + k) % kTaRows, tl = r / a.G;
    __nv_bfloat16* o = a.out + (static_cast<size_t>(first_row + tile * a.Tt + tl) * a.Hq + kvh * a.G + (r - tl * a.G)) * D + lane * kPer;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int j = 0; j < kPer; j += 2) w[j / 2] = pack_bf16x2(acc[k][j] * inv, acc[k][j + 1] * inv);
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(o) = w[0];
  }
}

}  // namespace pkv
