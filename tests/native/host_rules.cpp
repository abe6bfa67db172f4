// Rules that kernels share with the host, for the CPU tests (no CUDA).
#include <map>
#include <utility>
#include <vector>

#include "stage_ring.h"
#include "tree_plan.cuh"

using namespace pkv;

extern "C" {

int stage_bars_count(void) { return kStageBars; }
unsigned stage_bar_of(unsigned n) { return stage_bar(n); }
unsigned stage_parity_of(unsigned n) { return stage_parity(n); }

// The drafted-tree attention's shares for these lengths (0: inactive), walked
// as its kernels do.  what[0]: shares, what[1]: items that are joined,
// what[2..4]: the first fault's share, sequence and KV head.  Returns 0, or
//   1  a share writes a place twice
//   2  the merge reads a place that no unit of this call wrote
//   3  ... that holds another item or other steps
//   4  an item's parts do not make up its steps
//   5  an item is not written exactly once
//   6  a bound names an inactive sequence
int tree_shares_check(const int* ctx, int B, int Hkv, int item_steps, int min_steps, int max_shares, int* what) {
  std::vector<long long> start(B + 1, 0);
  for (int b = 0; b < B; ++b) start[b + 1] = start[b] + tree_cost(ctx[b], item_steps, Hkv);
  const long long total = start[B];
  const int shares = tree_share_count(total, min_steps, max_shares);
  what[0] = shares;
  what[1] = 0;
  int fault = 0;
  auto say = [&](int code, int share, int b, int kvh) {
    if (fault == 0) fault = code, what[2] = share, what[3] = b, what[4] = kvh;
  };
  std::vector<TreeBound> bounds(shares + 1);
  for (int s = 0; s <= shares; ++s) {
    bounds[s] = tree_bound(s, shares, total, start.data(), B, Hkv, item_steps);
    if (bounds[s].b < B) bounds[s].ctx = ctx[bounds[s].b];
  }
  auto steps_of = [&](int b) { return (ctx[b] + kTreeTokens - 1) / kTreeTokens; };
  struct Part {
    int b, kvh, j0, n;
  };
  std::map<std::pair<int, int>, Part> places;      // (share, place)
  std::map<std::pair<int, int>, int> outputs;      // (b, kvh): times written
  for (int share = 0; share < shares; ++share) {   // the attention: one CTA per share
    const TreeBound at = bounds[share], end = bounds[share + 1];
    int b = at.b, kvh = at.kvh, j0 = at.step;
    bool first_unit = true;
    while (b < end.b || (b == end.b && (kvh < end.kvh || (kvh == end.kvh && j0 < end.step)))) {
      const int nt = steps_of(b);
      if (nt == 0) {
        ++b;
        continue;
      }
      const int n = (b == end.b && kvh == end.kvh ? end.step : nt) - j0;
      const int part = tree_unit_part(j0, n, nt, first_unit);
      first_unit = false;
      if (part == 0)
        ++outputs[{b, kvh}];
      else if (!places.insert({{share, part - 1}, Part{b, kvh, j0, n}}).second)
        say(1, share, b, kvh);
      j0 = 0;
      if (++kvh == Hkv) {
        kvh = 0;
        ++b;
      }
    }
  }
  for (int share = 0; share + 1 < shares; ++share) {  // the merge: one per share
    const TreeBound mine = bounds[share], next = bounds[share + 1];
    if (!tree_splits(mine, next, share, shares)) continue;
    int last = share + 1;
    while (last + 1 < shares && !tree_item_ends(next, bounds[last + 1])) ++last;
    int done = 0;
    for (int s = share; s <= last; ++s) {
      const auto it = places.find({s, s == share ? tree_split_place(mine, next) : 0});
      if (it == places.end()) {
        say(2, s, next.b, next.kvh);
      } else if (it->second.b != next.b || it->second.kvh != next.kvh || it->second.j0 != done) {
        say(3, s, next.b, next.kvh);
      } else {
        done += it->second.n;
      }
    }
    if (done != steps_of(next.b)) say(4, share, next.b, next.kvh);
    ++outputs[{next.b, next.kvh}];
    ++what[1];
  }
  for (int b = 0; b < B; ++b)
    for (int h = 0; h < Hkv; ++h)
      if (outputs[{b, h}] != (ctx[b] > 0 ? 1 : 0)) say(5, -1, b, h);
  for (int s = 0; s < shares; ++s)
    if (bounds[s].b < B && bounds[s].ctx == 0) say(6, s, bounds[s].b, bounds[s].kvh);
  return fault;
}
}
