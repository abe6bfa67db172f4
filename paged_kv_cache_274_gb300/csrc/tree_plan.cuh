// Work shares of the tcgen05 drafted-tree attention: what its planner writes and
// its attention and merge kernels read (without CUDA, so that the host can
// check that the three agree).
//
// The steps of all (sequence, KV head) items in a row are cut into shares.  An
// item that shares split leaves partials (m, l, O), at most two per share: its
// first unit's at place 0, a later one's at place 1.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PKV_PLAN_FN __host__ __device__ __forceinline__
#define PKV_PLAN_CALL inline __host__ __device__ __noinline__
#else
#define PKV_PLAN_FN inline
#define PKV_PLAN_CALL inline
#endif

namespace pkv {

constexpr int kTreeTokens = 128;  // tokens of a step

// Start of a share.
struct TreeBound {
  int b, kvh;  // item (b = batch, kvh = 0: the end)
  int step;    // step of the item (0: the share starts with the item)
  int ctx;     // the sequence's validated length
};

// Quotients of what mostly fits 32 bits, in one place.
PKV_PLAN_CALL long long plan_div(long long x, int d) {
  return (x >> 32) != 0 ? x / d : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(d));
}

// Cost of a sequence of c tokens, in steps: for every KV head its steps and
// item_steps for the item's start and output; 0 for an inactive one.
PKV_PLAN_FN long long tree_cost(int c, int item_steps, int Hkv) {
  return c == 0 ? 0 : static_cast<long long>((c + kTreeTokens - 1) / kTreeTokens + item_steps) * Hkv;
}

// Shares of at least min_steps steps.
PKV_PLAN_FN int tree_share_count(long long total, int min_steps, int max_shares) {
  const long long n = plan_div(total + min_steps - 1, min_steps);
  return static_cast<int>(n < max_shares ? n : max_shares);
}

// The sequence with start[b] <= pos < start[b + 1] (pos < total): it is active.
PKV_PLAN_FN int tree_find(const long long* start, int B, long long pos) {
  int lo = 0, hi = B - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid + 1] > pos) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Start of share s (s == shares: the end), without ctx.  start: the prefix sums
// of the costs.  Shares are equal in cost.  A boundary within `near` steps of
// an item's start or end moves there: the partial it would leave costs more
// than the imbalance.  A boundary always names the item that the share really
// starts with (the attention and the merge both go by it), so one that moves
// past a sequence's last item goes to the next active sequence.
PKV_PLAN_FN TreeBound tree_bound(int s, int shares, long long total, const long long* start, int B, int Hkv, int item_steps) {
  TreeBound r{B, 0, 0, 0};
  if (s >= shares) return r;
  const long long apart = plan_div(total, shares) / 4;
  const int near = apart < 2 ? static_cast<int>(apart) : 2;
  const long long pos = plan_div(total * s, shares);
  r.b = tree_find(start, B, pos);
  const long long in = pos - start[r.b], next = start[r.b + 1];
  const int cost = static_cast<int>(plan_div(next - start[r.b], Hkv)), nt = cost - item_steps;
  r.kvh = static_cast<int>(plan_div(in, cost));
  const int step = static_cast<int>(in - static_cast<long long>(r.kvh) * cost) - item_steps;
  if (step <= near) return r;
  if (nt - step > near) {
    r.step = step;
  } else if (++r.kvh == Hkv) {
    r.kvh = 0;
    r.b = next < total ? tree_find(start, B, next) : B;
  }
  return r;
}

// Which partial a unit of n of an item's nt steps from step j0 on leaves: 0
// (the unit is the whole item: none), else 1 + its place.
PKV_PLAN_FN int tree_unit_part(int j0, int n, int nt, bool first_of_share) {
  return (j0 == 0 && n == nt) ? 0 : (first_of_share ? 1 : 2);
}

// Whether share `share` (from `mine` to `next`) leaves an item that it starts
// and others end, i.e. whose parts are joined in its name.
PKV_PLAN_FN bool tree_splits(const TreeBound& mine, const TreeBound& next, int share, int shares) {
  if (share + 1 >= shares) return false;  // the last share splits nothing
  if (next.step == 0) return false;       // an item starts there
  return !(mine.b == next.b && mine.kvh == next.kvh && mine.step > 0);
}
// Place of that share's part: its first unit's if it starts with the item.  (The
// parts of the shares after it are their first units'.)
PKV_PLAN_FN int tree_split_place(const TreeBound& mine, const TreeBound& next) {
  return mine.b == next.b && mine.kvh == next.kvh ? 0 : 1;
}
// Whether the item `at` ends with the share that ends where `e` is.
PKV_PLAN_FN bool tree_item_ends(const TreeBound& at, const TreeBound& e) {
  return e.b != at.b || e.kvh != at.kvh || e.step == 0;
}

}  // namespace pkv
