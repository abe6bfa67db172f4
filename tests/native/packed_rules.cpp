// The work shares of the attention of packed rows, walked as its kernels do
// (no CUDA).
#include <map>
#include <tuple>
#include <utility>
#include <vector>

#include "packed_plan.cuh"

using namespace pkv;

extern "C" {

// Sequences of ctx[b] cached tokens with m[b] rows.  what[0]: shares, what[1]:
// items that are joined, what[2..5]: the first fault's share, sequence, KV head
// and run; what[6], what[7]: least and most steps of a share.  Returns 0, or
//   1  a share writes a place twice
//   2  the merge reads a place that no unit of this call wrote
//   3  ... that holds another item or other steps
//   4  an item's parts do not make up its steps
//   5  an item with steps is not written exactly once, or one without is
//   6  a bound names no item, or a step outside it
//   7  a unit has no steps
//   8  more shares, or places of a share, than the workspace has
int packed_shares_check(const int* ctx, const int* m, int B, int Hkv, int span, int tile, int alone, int item_steps, int min_steps, int max_shares,
                        int* what) {
  std::vector<PackedSeq> seqs(B + 1);
  int row = 0;
  for (int b = 0; b < B; ++b) {
    seqs[b] = PackedSeq{ctx[b], row, m[b], 0};
    row += m[b];
  }
  std::vector<long long> start(B + 1, 0);
  const long long item_cost = packed_item_cost(item_steps);
  for (int b = 0; b < B; ++b) start[b + 1] = start[b] + packed_cost(seqs[b], span, item_cost) * packed_weight(seqs[b], tile, alone) * Hkv;
  const long long total = start[B];
  const int shares = packed_share_count(total, min_steps, max_shares);
  what[0] = shares;
  what[1] = 0;
  what[6] = 1 << 30;
  what[7] = 0;
  int fault = 0;
  auto say = [&](int code, int share, int b, int kvh, int run) {
    if (fault == 0) fault = code, what[2] = share, what[3] = b, what[4] = kvh, what[5] = run;
  };
  if (shares > max_shares) say(8, 0, 0, 0, 0);
  std::vector<PackedBound> bounds(shares + 1);
  for (int s = 0; s <= shares; ++s) {
    bounds[s] = packed_bound(s, shares, total, start.data(), seqs.data(), B, Hkv, span, tile, alone, item_steps);
    const PackedBound& x = bounds[s];
    if (x.b < B) {
      const PackedSeq& q = seqs[x.b];
      const bool item = q.ctx > 0 && q.m > 0 && x.kvh >= 0 && x.kvh < Hkv && x.run >= packed_first(q, span) && x.run < packed_runs(q, span);
      if (!item || x.step < 0 || x.step >= packed_steps(packed_seen(q, x.run, span))) say(6, s, x.b, x.kvh, x.run);
    } else if (x.kvh != 0 || x.run != 0 || x.step != 0) {
      say(6, s, x.b, x.kvh, x.run);
    }
  }
  if (fault) return fault;
  using Item = std::tuple<int, int, int>;
  struct Part {
    Item item;
    int j0, n;
  };
  std::map<std::pair<int, int>, Part> places;  // (share, place)
  std::map<Item, int> outputs;                 // times written
  for (int share = 0; share < shares; ++share) {  // the attention: one CTA per share
    const PackedBound at = bounds[share], end = bounds[share + 1];
    int b = at.b, kvh = at.kvh, run = at.run, j0 = at.step, steps = 0;
    bool first_unit = true;
    while (packed_is_before(b, kvh, run, j0, end)) {
      const PackedSeq seq = seqs[b];
      if (seq.ctx > 0 && seq.m > 0 && run < packed_first(seq, span)) run = packed_first(seq, span);
      if (!packed_is_before(b, kvh, run, j0, end)) break;
      const int seen = seq.ctx > 0 && seq.m > 0 ? packed_seen(seq, run, span) : 0;
      const int nt = packed_steps(seen);
      if (nt == 0) {
        ++b;
        run = 0;
        continue;
      }
      const int n = (b == end.b && kvh == end.kvh && run == end.run ? end.step : nt) - j0;
      if (n <= 0) say(7, share, b, kvh, run);
      const int part = tree_unit_part(j0, n, nt, first_unit);
      first_unit = false;
      steps += n;
      if (part == 0)
        ++outputs[Item{b, kvh, run}];
      else if (part > 2)
        say(8, share, b, kvh, run);
      else if (!places.insert({{share, part - 1}, Part{Item{b, kvh, run}, j0, n}}).second)
        say(1, share, b, kvh, run);
      j0 = 0;
      if (++run < packed_runs(seq, span)) continue;
      run = 0;
      if (++kvh == Hkv) {
        kvh = 0;
        ++b;
      }
    }
    if (steps < what[6]) what[6] = steps;
    if (steps > what[7]) what[7] = steps;
  }
  for (int share = 0; share + 1 < shares; ++share) {  // the merge: one per share
    const PackedBound mine = bounds[share], next = bounds[share + 1];
    if (!packed_splits(mine, next, share, shares)) continue;
    int last = share + 1;
    while (last + 1 < shares && !packed_item_ends(next, bounds[last + 1])) ++last;
    int done = 0;
    const Item item{next.b, next.kvh, next.run};
    for (int s = share; s <= last; ++s) {
      const auto it = places.find({s, s == share ? packed_split_place(mine, next) : 0});
      if (it == places.end()) {
        say(2, s, next.b, next.kvh, next.run);
      } else if (it->second.item != item || it->second.j0 != done) {
        say(3, s, next.b, next.kvh, next.run);
      } else {
        done += it->second.n;
      }
    }
    if (done != packed_steps(packed_seen(seqs[next.b], next.run, span))) say(4, share, next.b, next.kvh, next.run);
    ++outputs[item];
    ++what[1];
  }
  for (int b = 0; b < B; ++b)
    for (int h = 0; h < Hkv; ++h)
      for (int run = 0; run < packed_runs(seqs[b], span); ++run) {
        const bool steps = seqs[b].ctx > 0 && packed_seen(seqs[b], run, span) > 0;
        const auto it = outputs.find(Item{b, h, run});
        if ((it == outputs.end() ? 0 : it->second) != (steps ? 1 : 0)) say(5, -1, b, h, run);
      }
  return fault;
}
}
