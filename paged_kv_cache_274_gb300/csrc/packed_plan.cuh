// Work shares of the tcgen05 attention of packed rows: what its planner writes
// and its attention and merge kernels read (without CUDA, so that the host can
// check that the three agree).
//
// Sequence b has m rows, the last of its ctx cached tokens; row t sees the
// positions up to ctx - m + t.  An item is a run of `span` rows (the row tiles
// of a CTA) on one KV head; it takes the steps of the positions that its last
// row sees.  The items of all sequences in a row (sequence, KV head, rows) are
// cut into shares of equal cost, as the drafted trees' are (tree_plan.cuh); a
// split item's parts have the same places.
#pragma once

#include "tree_plan.cuh"

namespace pkv {

// A sequence's validated numbers.
struct PackedSeq {
  int ctx;    // cached tokens (0: none; its rows are zeros)
  int start;  // its first row
  int m;      // its rows (0: none to attend with)
  int unused;
};

// Start of a share.
struct PackedBound {
  int b, kvh, run;  // item (b = batch, kvh = run = 0: the end)
  int step;         // step of the item (0: the share starts with the item)
};

// Sequences' rows as the caller gives them.  Where an entry of query_starts lies
// below the one before it, that sequence and every one behind it are refused
// (`fall`: the first such sequence, or B): their rows could be others' too.
// Before it the entries rise, so the rows are their own, and a row's sequence is
// found among them by bisection.
PKV_PLAN_FN bool packed_falls(const int32_t* starts, int b) { return starts[b + 1] < starts[b]; }
// Whether the rows s0 .. s1 - 1 of sequence b can be served, of N rows, T a sequence at most.
PKV_PLAN_FN bool packed_rows_fit(int s0, int s1, int b, int fall, int N, int T) {
  return b < fall && s0 >= 0 && s0 <= s1 && s1 <= N && s1 - s0 <= T;
}
// The one sequence that `row` can belong to (-1: none).
PKV_PLAN_FN int packed_owner(const int32_t* starts, int fall, int row) {
  int lo = 0, hi = fall;  // the first sequence that starts behind the row
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] > row) hi = mid; else lo = mid + 1;
  }
  return lo - 1;
}

PKV_PLAN_FN int packed_runs(const PackedSeq& s, int span) { return (s.m + span - 1) / span; }

// Positions that the last row of a run sees (0: none of its rows sees any).
PKV_PLAN_FN int packed_seen(const PackedSeq& s, int run, int span) {
  const int rows = s.m - run * span < span ? s.m : (run + 1) * span;  // up to the run's end
  const int n = s.ctx - s.m + rows;
  return n > 0 ? n : 0;
}

PKV_PLAN_FN int packed_steps(int seen) { return (seen + kTreeTokens - 1) / kTreeTokens; }

// First run with a position to see (of a sequence with ctx > 0): with more rows
// than cached tokens, the first rows see none.
PKV_PLAN_FN int packed_first(const PackedSeq& s, int span) { return s.ctx >= s.m ? 0 : (s.m - s.ctx) / span; }

// Cost in tokens x kPackedWeight: what an item's last row sees, half a step of
// rounding, and item_steps for its start and output.  The items of a sequence
// whose rows fit one tile, where CTAs serve pairs of them, weigh `alone` in the
// place of kPackedWeight: their steps take half of the products.
constexpr int kPackedWeight = 8;
PKV_PLAN_FN long long packed_item_cost(int item_steps) { return kTreeTokens * static_cast<long long>(item_steps) + kTreeTokens / 2; }
PKV_PLAN_FN int packed_weight(const PackedSeq& s, int tile, int alone) { return s.m <= tile ? alone : kPackedWeight; }

// Of the first x items of a KV head, as if the last run were full.
PKV_PLAN_FN long long packed_before(const PackedSeq& s, long long x, int span, long long item_cost) {
  const long long one = static_cast<long long>(s.ctx) - s.m + static_cast<long long>(packed_first(s, span) + 1) * span + item_cost;
  return x * one + span * (x * (x - 1) / 2);
}

// Of a KV head of a sequence, unweighted.
PKV_PLAN_FN long long packed_cost(const PackedSeq& s, int span, long long item_cost) {
  if (s.ctx == 0 || s.m == 0) return 0;
  const int runs = packed_runs(s, span);
  return packed_before(s, runs - packed_first(s, span), span, item_cost) - (static_cast<long long>(runs) * span - s.m);
}

// Most shares of a call: a CTA each, which holds an SM alone, so no more than there
// are SMs (the others would run behind them, as long again).  The workspace has
// room for kPackedShares.
constexpr int kPackedShares = 152;
PKV_PLAN_FN int packed_most_shares(int num_sms) { return num_sms < kPackedShares ? (num_sms < 1 ? 1 : num_sms) : kPackedShares; }

// Shares of at least min_steps steps (never less than one: two boundaries in
// one step would leave a share inside an item without steps).
PKV_PLAN_FN int packed_share_count(long long total, int min_steps, int max_shares) {
  const long long n = total / (static_cast<long long>(min_steps) * kTreeTokens * kPackedWeight);
  return total == 0 ? 0 : n < 1 ? 1 : static_cast<int>(n < max_shares ? n : max_shares);
}

// Start of share s (s == shares: the end).  start: the prefix sums of the
// sequences' weighted costs (all KV heads).  A boundary within `near` steps of an item's
// start or end moves there.
PKV_PLAN_FN PackedBound packed_bound(int s, int shares, long long total, const long long* start, const PackedSeq* seqs, int B, int Hkv,
                                     int span, int tile, int alone, int item_steps) {
  PackedBound r{B, 0, 0, 0};
  if (s >= shares) return r;
  const long long apart = total / shares / (4 * kTreeTokens * kPackedWeight), item_cost = packed_item_cost(item_steps);
  const int near = apart < 2 ? static_cast<int>(apart) : 2;
  // (total * s may pass 64 bits)
  const long long pos = total / shares * s + total % shares * s / shares;
  r.b = tree_find(start, B, pos);
  const PackedSeq q = seqs[r.b];
  const int weight = packed_weight(q, tile, alone);
  const long long cost = (start[r.b + 1] - start[r.b]) / Hkv, in = pos - start[r.b];
  r.kvh = static_cast<int>(in / cost);
  const long long rest = (in - r.kvh * cost) / weight;
  const int first = packed_first(q, span), runs = packed_runs(q, span);
  int lo = 0, hi = runs - first - 1;  // the last item that starts at or before `rest`
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (packed_before(q, mid, span, item_cost) <= rest) lo = mid; else hi = mid - 1;
  }
  r.run = first + lo;
  const long long off = rest - packed_before(q, lo, span, item_cost) - item_cost;
  const int step = off <= 0 ? 0 : static_cast<int>(off / kTreeTokens);
  if (step <= near) return r;
  if (packed_steps(packed_seen(q, r.run, span)) - step > near) {
    r.step = step;
  } else if (++r.run == runs) {
    r.run = first;
    if (++r.kvh == Hkv) {
      r.kvh = 0;
      const long long next = start[r.b + 1];
      r.b = next < total ? tree_find(start, B, next) : B;
      r.run = r.b < B ? packed_first(seqs[r.b], span) : 0;
    }
  }
  return r;
}

PKV_PLAN_FN bool packed_same_item(const PackedBound& x, const PackedBound& y) { return x.b == y.b && x.kvh == y.kvh && x.run == y.run; }

// What the merge joins in a share's name (of the share in which the item starts).
struct PackedMerge {
  int parts;   // 0: nothing
  int place;   // of the share's own part; the others' are their first units'
  int row0;    // first row of the item
  int rows;    // rows of the sequence from there on
  int kvh;
  int unused[3];
};

// Whether the place (b, kvh, run, step) lies before `end`.
PKV_PLAN_FN bool packed_is_before(int b, int kvh, int run, int step, const PackedBound& end) {
  if (b != end.b) return b < end.b;
  if (kvh != end.kvh) return kvh < end.kvh;
  if (run != end.run) return run < end.run;
  return step < end.step;
}

// As tree_splits, tree_split_place and tree_item_ends.
PKV_PLAN_FN bool packed_splits(const PackedBound& mine, const PackedBound& next, int share, int shares) {
  if (share + 1 >= shares || next.step == 0) return false;
  return !(packed_same_item(mine, next) && mine.step > 0);
}
PKV_PLAN_FN int packed_split_place(const PackedBound& mine, const PackedBound& next) { return packed_same_item(mine, next) ? 0 : 1; }
PKV_PLAN_FN bool packed_item_ends(const PackedBound& at, const PackedBound& e) { return !packed_same_item(at, e) || e.step == 0; }

}  // namespace pkv
