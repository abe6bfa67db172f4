// Verification of drafted trees against the target model's probabilities, from
// given random numbers.
//
// The walk starts at the root.  At a node u with target row p and draft row q
// (both over the vocabulary) the children c, tokens x_c, are tried in order,
// with P = p, Q = q, Z = Y = 1 at first:
//   accept c if r_c Q(x_c) / Y < P(x_c) / Z, and go on from c;
//   else P = max(P - (Z / Y) Q, 0), Q(x_c) = 0, Z = sum P, Y = sum Q.
// Where no child is accepted, the next token is drawn from P / Z: the first j
// whose partial sum of P exceeds u Z.  (That leaves the target's distribution,
// for children drawn one after another without replacement from q; without q, Q
// is 1 at x_c and 0 elsewhere: children that were chosen without randomness.)
//
// Since q >= 0, the rounds at one node join: P = max(p - A q, 0) with A the sum
// of the rounds' Z / Y, so a round is one pass over p and q that needs nothing
// but A, and a removed token's P is 0 by itself.  Where Y is next to nothing (a
// draft row with all but 1e-30 of its weight on a rejected token), A would leave
// fp32's range: it is kept as -A 2^-64 then, and multiplies -q 2^64.
//
// The drawn token is a border among sums over the vocabulary, so everything is
// summed to 2^-32 or better: p - A q is kept as an unevaluated sum of two
// floats (error-free transformations of addition and product, T. J. Dekker and
// D. E. Knuth), so is everything that is summed or compared.  (A is right to some
// 2^-46, so p - A q to 2^-44 of A q where a node loses two children or more; behind
// the first it is exact.)  There are no
// doubles in it: fp64 units do 2 operations a clock and SM, and with doubles in the
// draw alone it took 9 to 12 us of a call instead of 2.  (Only a comparison whose
// products leave fp32's range is made of doubles.)
//
// What bounds it: the rows of the nodes where the walk loses a child or ends,
// from HBM, and for a small batch the chain of loads.  One cluster of up to 16
// CTAs per sequence.  Its first CTA walks (a warp; the nodes' own p and q are
// gathered beforehand, side by side) and tells the others by distributed shared
// memory which row to sum next; the CTAs take its chunks of 512 values in turn.
// Only the first CTA decides, so the others cannot come to another end.
//
// Measured: 64 sequences, 32 nodes, 128,256 tokens, drawn drafts 44 to 47 us (1.75 passes
// a sequence on average, 5 or 6 in the slowest: the first from HBM together, 7 to 10
// us, then a few sequences' in turn, each 3.7 us of sums, a chunk's latency from L2 at
// a time, 2.2 of a cluster barrier and the first warp's decision and 0.7 of the other
// barrier; 4 us at the end for the draw); 48 sequences, 21 nodes, 50,257 tokens,
// drafts without randomness 15 to 18 us (a pass at each node that loses a child); one
// sequence, 8 nodes, 32,000 tokens 8 to 19 us, by its passes.  Kept one by one for
// the batch: the copies ahead 54 -> 48, two elements an instruction 46.4 -> 43.8.
// (Later chunks prefetched to L2 at a pass's start: 58 instead of 54; the first chunk
// by loads and the second copied beside it: 66, with 600 bytes of registers spilt.)
#include <algorithm>

#include <cooperative_groups.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyChunk = 512;  // values that a warp sums at a time
constexpr int kPer = kVerifyChunk / 32;
constexpr int kVerifyMaxChunks = (PKV_MAX_VOCAB + 3 + kVerifyChunk - 1) / kVerifyChunk;
// From Y below this much of Z on, A is kept times -2^-64 and q times -2^64.  (Y is
// 2^-149 or more, so A is at most 2^149 Z; the q that are left are below Y.)
constexpr float kVerifyLeastY = 0x1p-100f;
constexpr float kVerifyRaise = -0x1p64f;
constexpr int kVerifyCluster = 16;  // most CTAs of a cluster (more than 8 by a launch attribute of the kernel)

// An unevaluated sum hi + lo.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// hi takes what it can hold of the sum (|hi| >= |lo|).
__device__ __forceinline__ Pair joined(float hi, float lo) {
  const float s = __fadd_rn(hi, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ void add_to(Pair& x, const Pair& y) {
  const Pair s = two_sum(x.hi, y.hi);
  x = joined(s.hi, __fadd_rn(s.lo, __fadd_rn(x.lo, y.lo)));
}
__device__ __forceinline__ Pair times(const Pair& x, const Pair& y) {
  const float h = __fmul_rn(x.hi, y.hi);
  return joined(h, fmaf(x.lo, y.hi, fmaf(x.hi, y.lo, fmaf(x.hi, y.hi, -h))));
}
// x / y in two steps of long division
__device__ __forceinline__ Pair over(const Pair& x, const Pair& y) {
  const float q = __fdiv_rn(x.hi, y.hi);
  const Pair p = times(y, Pair{q, 0.f}), d = two_sum(x.hi, -p.hi);
  return joined(q, __fdiv_rn(__fadd_rn(d.hi, __fadd_rn(d.lo, __fsub_rn(x.lo, p.lo))), y.hi));
}
// (of joined pairs)
__device__ __forceinline__ bool below(const Pair& x, const Pair& y) { return x.hi < y.hi || (x.hi == y.hi && x.lo < y.lo); }
// x times a power of two
__device__ __forceinline__ Pair scaled(const Pair& x, float f) { return {__fmul_rn(x.hi, f), __fmul_rn(x.lo, f)}; }
__device__ __forceinline__ double whole(const Pair& x) { return static_cast<double>(x.hi) + x.lo; }
__device__ __forceinline__ bool positive(const Pair& x) { return x.hi > 0.f || (x.hi == 0.f && x.lo > 0.f); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// What is negative or not finite counts as 0.  (The bits of those, and of -0, are
// at least infinity's.)
__device__ __forceinline__ float clean(float x) { return __float_as_uint(x) < 0x7f800000u ? x : 0.f; }
__device__ __forceinline__ Pair weight(float p) { return {clean(p), 0.f}; }
// max(p - (ah + al) q, 0), likewise.  (Where p >= ah q, three operations give
// the difference and what it rounds away; elsewhere the result is 0.  It is 0 by
// itself for p < 0, and for p that is not finite: d + lo is NaN then.)
__device__ __forceinline__ Pair weight_left(float p, float q, float ah, float al) {
  q = clean(q);
  const float h = __fmul_rn(ah, q);
  const float l = fmaf(al, q, fmaf(ah, q, -h));
  const float d = __fsub_rn(p, h);
  const float lo = __fsub_rn(__fsub_rn(__fsub_rn(p, d), h), l);
  const bool some = __fadd_rn(d, lo) > 0.f;
  return {some ? d : 0.f, some ? lo : 0.f};
}
// -q times kVerifyRaise, finite (a rejected token's may be anything; it takes all of
// P as the largest number does).
__device__ __forceinline__ float raised(float q) { return fminf(__fmul_rn(clean(q), -kVerifyRaise), 0x1.fffffep127f); }
__device__ __forceinline__ Pair warp_total(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair y{__shfl_xor_sync(kFull, x.hi, o), __shfl_xor_sync(kFull, x.lo, o)};
    add_to(x, y);
  }
  return x;
}
// Of two, side by side.
__device__ __forceinline__ void warp_totals(Pair& x, Pair& y) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair u{__shfl_xor_sync(kFull, x.hi, o), __shfl_xor_sync(kFull, x.lo, o)};
    const Pair v{__shfl_xor_sync(kFull, y.hi, o), __shfl_xor_sync(kFull, y.lo, o)};
    add_to(x, u);
    add_to(y, v);
  }
}

struct VerifyShared {
  // what to sum next, written by the cluster's first CTA
  int row;       // of the sequence; -1: nothing more
  int removed;   // tokens in `gone`
  int want_y;
  int last;      // the walk ends with these sums: only its warp goes on
  float ah, al;
  Pair y_part[kVerifyCluster * kVerifyWarps];  // (first CTA)
  int gone[PKV_MAX_QUERY_TOKENS];              // tokens of the rejected children
  // the nodes (first CTA)
  int token[PKV_MAX_QUERY_TOKENS], parent[PKV_MAX_QUERY_TOKENS];
  float r[PKV_MAX_QUERY_TOKENS], p[PKV_MAX_QUERY_TOKENS], q[PKV_MAX_QUERY_TOKENS];
  union {
    // the next chunk of a warp's pass, p and q, on its way
    alignas(16) float stage[kVerifyWarps][2][kVerifyChunk];
    Pair weights[kVerifyChunk / 16 * 17];  // of the chunk that the token is drawn from (verify_pad)
  };
};

// Rows start at any float.  Their chunks are counted from the 16-byte boundary
// before them, `shift` floats back, so that a lane's four values are one load;
// with a draft row on another shift they are single loads (shift 0).
struct VerifyRows {
  const float* p;
  const float* q;  // NULL: no draft row
  int shift;
  bool vec;
};
// draft: the draft row counts (a child was rejected).
__device__ __forceinline__ VerifyRows verify_rows(const VerifyArgs& a, size_t row, bool draft) {
  VerifyRows r;
  r.p = a.p + row * a.p_stride;
  r.q = draft && a.q != nullptr ? a.q + row * a.q_stride : nullptr;
  const int sp = static_cast<int>(reinterpret_cast<uintptr_t>(r.p) >> 2) & 3;
  r.vec = r.q == nullptr || (static_cast<int>(reinterpret_cast<uintptr_t>(r.q) >> 2) & 3) == sp;
  r.shift = r.vec ? sp : 0;
  return r;
}

// A chunk's values, 16 a lane: lane's value k is at e0 + verify_at(k, lane).
__device__ __forceinline__ int verify_at(int k, int lane) { return (k / 4) * 128 + lane * 4 + k % 4; }
// (0 outside the row)
__device__ __forceinline__ void verify_load(float (&x)[kPer], const float* row, int e0, int V, int lane, bool vec) {
#pragma unroll
  for (int k = 0; k < kPer; k += 4) {
    const int e = e0 + verify_at(k, lane);
    if (vec && e >= 0 && e + 4 <= V) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + e));
      x[k] = v.x;
      x[k + 1] = v.y;
      x[k + 2] = v.z;
      x[k + 3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[k + j] = e + j >= 0 && e + j < V ? __ldg(row + e + j) : 0.f;
    }
  }
}

// 0 for the rejected children's tokens.
__device__ __forceinline__ void verify_drop(float (&x)[kPer], const VerifyShared* s, int removed, int e0, int lane) {
#pragma unroll 1
  for (int g = 0; g < removed; ++g) {
    const int d = s->gone[g] - e0;
    if (static_cast<unsigned>(d) < static_cast<unsigned>(kVerifyChunk)) {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (verify_at(k, lane) == d) x[k] = 0.f;
    }
  }
}

// Two floats a register pair: one instruction rounds both as it would each.
using F2 = uint64_t;
__device__ __forceinline__ F2 both(float x, float y) { return static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x); }
__device__ __forceinline__ float first(F2 x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float second(F2 x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ F2 add2(F2 x, F2 y) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 x, F2 y) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 x, F2 y, F2 z) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}
__device__ __forceinline__ F2 sub2(F2 x, F2 y) { return fma2(y, both(-1.f, -1.f), x); }

// Two unevaluated sums.
struct Pairs {
  F2 hi, lo;
};
// weight_left of two elements, q cleaned.
__device__ __forceinline__ Pairs weights_left(F2 p, F2 q, float ah, float al) {
  const F2 nh = mul2(both(-ah, -ah), q);
  const F2 l = fma2(both(al, al), q, fma2(both(ah, ah), q, nh));
  const F2 d = add2(p, nh);
  const F2 lo = sub2(add2(sub2(p, d), nh), l), v = add2(d, lo);
  const bool some0 = first(v) > 0.f, some1 = second(v) > 0.f;
  return {both(some0 ? first(d) : 0.f, some1 ? second(d) : 0.f), both(some0 ? first(lo) : 0.f, some1 ? second(lo) : 0.f)};
}

// Sum of a lane's values, at(k) those of k and k + 1, four running sums side by
// side.  Each keeps what its additions round away in `lo`.  PARTS: the values
// have low parts.
template <bool PARTS, typename F>
__device__ __forceinline__ Pair verify_sum(F&& at) {
  Pairs s[2];
#pragma unroll
  for (int k = 0; k < kPer; k += 2) {
    const Pairs w = at(k);
    Pairs& t = s[k / 2 % 2];
    if (k < 4) {
      t = w;
    } else {
      const F2 a = t.hi, sum = add2(a, w.hi), u = sub2(sum, a);
      F2 lost = add2(sub2(a, sub2(sum, u)), sub2(w.hi, u));
      if (PARTS) lost = add2(lost, w.lo);
      t = {sum, add2(t.lo, lost)};
    }
  }
  Pair x{first(s[0].hi), first(s[0].lo)}, y{first(s[1].hi), first(s[1].lo)};
  add_to(x, Pair{second(s[0].hi), second(s[0].lo)});
  add_to(y, Pair{second(s[1].hi), second(s[1].lo)});
  add_to(x, y);
  return x;
}
// Of plain weights.
__device__ __forceinline__ Pair verify_sum_of(const float (&x)[kPer]) {
  return verify_sum<false>([&](int k) { return Pairs{both(clean(x[k]), clean(x[k + 1])), 0ull}; });
}

// Sum of chunk i of the target's weights without the removed tokens.
__device__ __noinline__ Pair verify_chunk_alone(const VerifyArgs& a, const VerifyShared* s, const VerifyRows& r, int i, int removed) {
  const int lane = threadIdx.x & 31, e0 = i * kVerifyChunk - r.shift;
  float pv[kPer];
  verify_load(pv, r.p, e0, a.V, lane, r.vec);
  verify_drop(pv, s, removed, e0, lane);
  return warp_total(verify_sum_of(pv));
}

// A lane's 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy_16(float* to, const float* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

// This CTA's chunks of the row: sums of max(p - A q, 0) to the first CTA's
// `sums`, this warp's sum of the Q that are left to its y_part.  A warp's next
// chunk is on its way to shared memory while it sums one; each lane reads what
// it copied itself.
template <bool DRAFT>
__device__ __forceinline__ void verify_pass(const VerifyArgs& a, VerifyShared* s, Pair* sums0, Pair* y_part0, const VerifyRows& r,
                                            int rank, int ranks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float ah = s->ah, al = s->al;
  const int removed = s->removed, chunks = (a.V + r.shift + kVerifyChunk - 1) / kVerifyChunk, apart = kVerifyWarps * ranks;
  const bool want_y = s->want_y != 0;
  float* p_stage = s->stage[warp][0] + 4 * lane;
  float* q_stage = s->stage[warp][1] + 4 * lane;
  // whole chunks of aligned rows are copied, others loaded when their turn comes
  auto copied = [&](int i) { return r.vec && i * kVerifyChunk >= r.shift && (i + 1) * kVerifyChunk - r.shift <= a.V; };
  auto fetch = [&](int i) {
    if (i < chunks && copied(i)) {
      const int e = i * kVerifyChunk - r.shift + 4 * lane;
#pragma unroll
      for (int k = 0; k < kVerifyChunk; k += 128) {
        copy_16(p_stage + k, r.p + e + k);
        if constexpr (DRAFT) copy_16(q_stage + k, r.q + e + k);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto take = [&](float (&x)[kPer], const float* from) {
#pragma unroll
    for (int k = 0; k < kPer; k += 4) {
      const float4 v = *reinterpret_cast<const float4*>(from + 32 * k);
      x[k] = v.x;
      x[k + 1] = v.y;
      x[k + 2] = v.z;
      x[k + 3] = v.w;
    }
  };
  Pair y{0.f, 0.f}, held{0.f, 0.f};  // the lane's part of the chunk before
  int held_at = -1;
  fetch(warp * ranks + rank);
#pragma unroll 1
  for (int i = warp * ranks + rank; i < chunks; i += apart) {
    const int e0 = i * kVerifyChunk - r.shift;
    float pv[kPer];
    [[maybe_unused]] float qv[kPer];
    if (held_at >= 0) {  // (while the copies are on their way)
      const Pair z = warp_total(held);
      if (lane == 0) sums0[held_at] = z;
    }
    held_at = i;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (copied(i)) {
      take(pv, p_stage);
      if constexpr (DRAFT) take(qv, q_stage);
    } else {
      verify_load(pv, r.p, e0, a.V, lane, r.vec);
      if constexpr (DRAFT) verify_load(qv, r.q, e0, a.V, lane, r.vec);
    }
    __syncwarp();  // (read before it is written again)
    fetch(i + apart);
    if constexpr (!DRAFT) {
      verify_drop(pv, s, removed, e0, lane);
      held = verify_sum_of(pv);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) qv[k] = clean(qv[k]);
      if (ah < 0.f) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) qv[k] *= kVerifyRaise;
      }
      held = verify_sum<true>([&](int k) { return weights_left(both(pv[k], pv[k + 1]), both(qv[k], qv[k + 1]), ah, al); });
      if (want_y) {
        verify_drop(qv, s, removed, e0, lane);
        Pair left = verify_sum<false>([&](int k) { return Pairs{both(qv[k], qv[k + 1]), 0ull}; });
        if (ah < 0.f) left = scaled(left, 1.f / kVerifyRaise);
        add_to(y, left);
      }
    }
  }
  warp_totals(held, y);
  if (lane == 0) {
    if (held_at >= 0) sums0[held_at] = held;
    if (want_y) y_part0[rank * kVerifyWarps + warp] = y;
  }
}

// r q Z < left Y where the products, or their low parts, may leave fp32's range.
__device__ __noinline__ bool verify_accepts(float r, float q, Pair left, Pair Y, Pair Z) {
  return static_cast<double>(r) * q * whole(Z) < whole(left) * whole(Y);
}

// Inclusive scan over the warp.  (Not inlined: code that runs once costs its
// fetch, 5 cycles and more an instruction.)
__device__ __noinline__ Pair warp_scan(Pair x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y{__shfl_up_sync(kFull, x.hi, o), __shfl_up_sync(kFull, x.lo, o)};
    Pair t = x;
    add_to(t, y);
    if (lane >= o) x = t;
  }
  return x;
}
__device__ __forceinline__ Pair from_lane(const Pair& x, int lane) { return {__shfl_sync(kFull, x.hi, lane), __shfl_sync(kFull, x.lo, lane)}; }
// What the lanes before this one have, of an inclusive scan.
__device__ __forceinline__ Pair warp_before(const Pair& upto) {
  const Pair y{__shfl_up_sync(kFull, upto.hi, 1), __shfl_up_sync(kFull, upto.lo, 1)};
  return (threadIdx.x & 31) > 0 ? y : Pair{0.f, 0.f};
}

// Sums of n pairs, a run of them per lane: up to each run's end.  One warp.
__device__ __forceinline__ int verify_run(int n) { return (n + 31) / 32; }
__device__ __forceinline__ Pair verify_lane_run(const Pair* x, int n) {
  const int per = verify_run(n), i0 = min((static_cast<int>(threadIdx.x) & 31) * per, n), i1 = min(i0 + per, n);
  Pair t{0.f, 0.f};
#pragma unroll 1
  for (int i = i0; i < i1; ++i) add_to(t, x[i]);
  return t;
}
__device__ __forceinline__ Pair verify_runs(const Pair* x, int n) { return warp_scan(verify_lane_run(x, n)); }

// A lane's 16 values in a row, without bank conflicts among the lanes.
__device__ __forceinline__ int verify_pad(int i) { return i + (i >> 4); }

// The first index whose partial sum exceeds `target` (the last with any weight,
// should rounding leave none); `upto`: verify_runs of the chunks.  One warp.
__device__ __forceinline__ int verify_draw(const VerifyArgs& a, VerifyShared* s, const Pair* sums, const VerifyRows& r, const Pair& A,
                                           int removed, const Pair& upto, const Pair& target) {
  const int lane = threadIdx.x & 31, chunks = (a.V + r.shift + kVerifyChunk - 1) / kVerifyChunk, per = verify_run(chunks);
  const Pair runs_before = warp_before(upto);
  unsigned found = __ballot_sync(kFull, below(target, upto));
  const bool last = found == 0;
  if (last) found = __ballot_sync(kFull, below(runs_before, upto));  // runs with any weight
  if (found == 0) return -1;
  const int run = last ? 31 - __clz(found) : __ffs(found) - 1, c1 = min((run + 1) * per, chunks);
  Pair base = from_lane(runs_before, run);
  int chunk = -1;
#pragma unroll 1
  for (int c = run * per; c < c1 && (last || chunk < 0); c += 32) {  // (once, up to 512k tokens)
    const Pair w = c + lane < c1 ? sums[c + lane] : Pair{0.f, 0.f};
    const Pair in = warp_scan(w);
    Pair at = base;
    add_to(at, in);
    unsigned m = __ballot_sync(kFull, positive(w) && (last || below(target, at)));
    if (m != 0) {
      const int k = last ? 31 - __clz(m) : __ffs(m) - 1;
      chunk = c + k;
      if (!last && k > 0) add_to(base, from_lane(in, k - 1));
    } else {
      add_to(base, from_lane(in, 31));
      m = __ballot_sync(kFull, positive(w));  // (kept, should the sums disagree in their last bits)
      if (m != 0 && !last && c + 32 >= c1) chunk = c + 31 - __clz(m);
    }
  }
  if (chunk < 0) return -1;
  // its weights, 16 in a row a lane
  const int e0 = chunk * kVerifyChunk - r.shift;
  {
    float pv[kPer], qv[kPer];
    verify_load(pv, r.p, e0, a.V, lane, r.vec);
    if (r.q != nullptr) verify_load(qv, r.q, e0, a.V, lane, r.vec);
#pragma unroll
    for (int k = 0; k < kPer; ++k) s->weights[verify_pad(verify_at(k, lane))] = Pair{pv[k], r.q != nullptr ? qv[k] : 0.f};
  }
  __syncwarp();
  if (r.q == nullptr)
#pragma unroll 1
    for (int g = lane; g < removed; g += 32)
      if (static_cast<unsigned>(s->gone[g] - e0) < static_cast<unsigned>(kVerifyChunk)) s->weights[verify_pad(s->gone[g] - e0)].hi = 0.f;
  __syncwarp();
  if (A.hi < 0.f)
#pragma unroll 1
    for (int k = 0; k < kPer; ++k) s->weights[verify_pad(lane * kPer + k)].lo = raised(s->weights[verify_pad(lane * kPer + k)].lo);
  const float ah = fabsf(A.hi), al = A.hi < 0.f ? -A.lo : A.lo;
  Pair own{0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < kPer; ++k) {
    Pair& w = s->weights[verify_pad(lane * kPer + k)];
    w = weight_left(w.hi, w.lo, ah, al);
    w = two_sum(w.hi, w.lo);  // (where p is near A q, the low part may be the larger)
    add_to(own, w);
  }
  __syncwarp();
  const Pair in = warp_scan(own), own_before = warp_before(in);
  Pair at = base;
  add_to(at, in);
  unsigned m = last ? 0u : __ballot_sync(kFull, below(target, at));
  const bool hit_lane = m != 0;
  if (!hit_lane) m = __ballot_sync(kFull, positive(own));
  if (m == 0) return -1;
  const int owner = hit_lane ? __ffs(m) - 1 : 31 - __clz(m);
  add_to(base, from_lane(own_before, owner));
  const Pair w = lane < kPer ? s->weights[verify_pad(owner * kPer + lane)] : Pair{0.f, 0.f};
  at = base;
  add_to(at, warp_scan(w));
  const bool any = positive(w);
  const int hit = hit_lane && any && below(target, at) ? e0 + owner * kPer + lane : -1, tail = any ? e0 + owner * kPer + lane : -1;
  const unsigned hits = __ballot_sync(kFull, hit >= 0);
  return hits != 0 ? __shfl_sync(kFull, hit, __ffs(hits) - 1) : __reduce_max_sync(kFull, tail);
}

__global__ void __launch_bounds__(kVerifyThreads, 4) verify_tree_kernel(const VerifyArgs a) {
  __shared__ VerifyShared s;
  extern __shared__ Pair sums[];  // (first CTA) of the chunks
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive();
  pdl_trigger();
  pdl_wait();
  const size_t seq = static_cast<size_t>(b) * a.T;
  auto row_p = [&](int t) { return a.p + (seq + t) * a.p_stride; };
  auto row_q = [&](int t) { return a.q + (seq + t) * a.q_stride; };

  // the nodes, and what the target and the draft give them
  int nodes = 0;
  bool bad = false;
  float u = 0.f;
  if (rank == 0) {
    u = a.sample_uniforms[b];
    nodes = a.node_counts != nullptr ? a.node_counts[b] : a.T;
    if (nodes < 0 || nodes > a.T) {
      bad = true;
      nodes = 0;
    }
    for (int t = tid; t < nodes; t += kVerifyThreads) {
      const int x = a.tokens[seq + t], u = a.parents[seq + t];
      s.token[t] = x;
      s.parent[t] = u;
      s.r[t] = a.accept_uniforms[seq + t];
      const bool fits = t == 0 ? u == -1 : u >= 0 && u < t && x >= 0 && x < a.V;
      bad |= !fits;
      if (t > 0 && fits) {
        s.p[t] = __ldg(row_p(u) + x);
        s.q[t] = a.q != nullptr ? __ldg(row_q(u) + x) : 1.f;
      }
    }
    bad = __syncthreads_or(bad) != 0;
    if (bad) nodes = 0;
  }

  // the walk's state (the first CTA's warp 0, the same in every lane)
  int at = 0, count = 0, next = 1, removed = 0, token = -1;
  const Pair none{0.f, 0.f}, one{1.f, 0.f};
  Pair A = none, Z = one, Y = one;
  bool summed = false;    // `sums` are those of P as it is
  Pair y_sum{-1.f, 0.f};  // Y as it was last summed (< 0: not at this node)
  Pair z_sum = none, upto = none;  // Z as it was last summed, and the runs' ends then
  bool stale = false;     // `sums` have changed since
  // Sums of P below this are nothing but what A and its products were rounded by (P
  // is 0 by the definition where it was a multiple of Q), or of a P that was nothing
  float least = 0.f;
  bool walking = nodes > 0, done = false;
  if (rank == 0 && warp == 0 && walking) {
    count = 1;
    if (lane == 0) a.accept_idx[static_cast<size_t>(b) * a.A] = 0;
  }
  auto child = [&](int from) {  // the next child of `at`, or -1
    for (int t0 = from; t0 < nodes; t0 += 32) {
      const unsigned m = __ballot_sync(kFull, t0 + lane < nodes && s.parent[min(t0 + lane, PKV_MAX_QUERY_TOKENS - 1)] == at);
      if (m != 0) return t0 + __ffs(m) - 1;
    }
    return -1;
  };
  // the first CTA's warp 0 tells every CTA what to sum
  auto tell = [&](int row, bool want_y, bool last) {
    if (lane < ranks) {
      VerifyShared* to = cluster.map_shared_rank(&s, lane);
      to->row = row;
      to->removed = removed;
      to->want_y = want_y ? 1 : 0;
      to->last = last ? 1 : 0;
      to->ah = A.hi;
      to->al = A.lo;
      if (removed > 0) to->gone[removed - 1] = s.token[next - 1];
    }
  };
  Pair* sums0 = cluster.map_shared_rank(sums, 0);
  Pair* y_part0 = cluster.map_shared_rank(s.y_part, 0);

  cluster_wait();  // every CTA of the cluster runs
  for (;;) {
    if (rank == 0 && warp == 0) {
      bool ask = false;
      while (walking && !ask) {
        const int c = count < a.A ? child(next) : -1;
        if (c < 0) {
          walking = false;
          break;
        }
        next = c + 1;
        const int x = s.token[c];
        bool was = false;  // its token was a rejected sibling's
        for (int g = lane; g < removed; g += 32) was |= s.gone[g] == x;
        was = __any_sync(kFull, was);
        const float q0 = weight(s.q[c]).hi;
        const Pair q{was && a.q != nullptr ? 0.f : q0, 0.f};
        Pair left = A.hi < 0.f ? weight_left(s.p[c], raised(q0), -A.hi, -A.lo) : weight_left(s.p[c], a.q != nullptr ? q0 : 0.f, A.hi, A.lo);
        left = was || !(Z.hi > 0.f) ? none : two_sum(left.hi, left.lo);
        const Pair rqz = times(times(Pair{s.r[c], 0.f}, q), Z), py = times(left, Y);
        bool accepted = below(rqz, py);
        if (left.hi > 0.f && !(fminf(rqz.hi, py.hi) >= 0x1p-70f && fmaxf(rqz.hi, py.hi) < 0x1p100f))
          accepted = verify_accepts(s.r[c], q.hi, left, Y, Z);
        if (accepted) {
          if (lane == 0) a.accept_idx[static_cast<size_t>(b) * a.A + count] = c;
          ++count;
          at = c;
          removed = 0;
          A = none;
          Z = Y = one;
          least = 0.f;
          y_sum.hi = -1.f;
          summed = false;
        } else {
          least = a.q == nullptr || Z.hi > 0.f ? 0.f : INFINITY;
          if (removed++ == 0)
            A = one;
          else if (a.q != nullptr && Y.hi > 0.f) {
            if (A.hi > 0.f && Y.hi < Z.hi * kVerifyLeastY) A = scaled(A, 1.f / kVerifyRaise);
            const Pair y = A.hi > 0.f ? Y : scaled(Y, kVerifyRaise);
            add_to(A, over(Z, y));
            // (where no token comes twice, P is a multiple of Q by chance alone)
            if (was) {
              const float rough = (__float_as_uint(A.hi) & 0x7fffffu) != 0u ? fabsf(A.hi) * 0x1p-46f : 0.f;
              least += fmaf(fmaf(fabsf(A.lo), 0x1p-22f, rough), fabsf(y.hi), Z.hi * 0x1p-44f);
            }
          }
          const bool more = count < a.A && child(next) >= 0;
          if (a.q == nullptr && summed) {
            // Only this token's chunk changes.  Summed anew where the difference
            // may be nothing but rounding, everything where Z has lost 8 bits.
            if (lane == 0) s.gone[removed - 1] = x;
            __syncwarp();
            if (!was && q0 > 0.f) {
              const VerifyRows r = verify_rows(a, seq + at, false);
              const int i = (x + r.shift) / kVerifyChunk;
              const float px = weight(s.p[c]).hi, whole_sum = sums[i].hi;
              Pair z = sums[i];
              add_to(z, Pair{-px, 0.f});
              if (!(z.hi > whole_sum * 0x1p-38f)) z = verify_chunk_alone(a, &s, r, i, removed);
              __syncwarp();
              if (lane == 0) sums[i] = z;
              __syncwarp();
              add_to(Z, Pair{-px, 0.f});
              stale = true;
            }
            if (!(Z.hi >= z_sum.hi / 256)) {
              for (int rr = 0; rr < ranks; ++rr)
                for (int g = lane; g < removed; g += 32) cluster.map_shared_rank(&s, rr)->gone[g] = s.gone[g];
              tell(at, false, !more);
              ask = true;
            }
          } else {
            // Y without this token: summed again only where the difference would
            // lose more than 8 bits
            bool want_y = false;
            if (a.q != nullptr && more) {
              add_to(Y, Pair{-q.hi, 0.f});
              want_y = !(y_sum.hi >= 0.f && Y.hi >= y_sum.hi / 256);
            }
            tell(at, want_y, !more);
            ask = true;
          }
        }
      }
      if (!ask && nodes > 0 && !summed) {  // the target's own weights
        tell(at, false, true);
        ask = true;
      }
      done = !ask;
      if (done) tell(-1, false, true);
      summed = true;
    }
    cluster_arrive();  // the request is there
    if (done) break;   // (the walking warp goes on, and waits when it is through)
    cluster_wait();
    const int row = s.row;
    if (row < 0) return;
    const VerifyRows r = verify_rows(a, seq + row, s.removed > 0);
    if (r.q != nullptr)
      verify_pass<true>(a, &s, sums0, y_part0, r, rank, ranks);
    else
      verify_pass<false>(a, &s, sums0, y_part0, r, rank, ranks);
    const bool last = s.last != 0;
    cluster_arrive();  // the sums are there
    if (last && (rank != 0 || warp != 0)) return;
    cluster_wait();
    if (rank == 0 && warp == 0) {
      const int n = (a.V + r.shift + kVerifyChunk - 1) / kVerifyChunk;
      stale = false;
      if (last) {
        upto = verify_runs(sums, n);
        z_sum = Z = from_lane(upto, 31);
        if (Z.hi < least) Z = none;
        break;
      }
      // (the runs' ends wait until a token is drawn)
      stale = true;
      Z = verify_lane_run(sums, n);
      Pair y = s.want_y ? verify_lane_run(s.y_part, ranks * kVerifyWarps) : none;
      warp_totals(Z, y);
      if (Z.hi < least) Z = none;
      z_sum = Z;
      if (s.want_y) y_sum = Y = y;
    }
  }
  if (nodes > 0) {
    VerifyRows r = verify_rows(a, seq + at, removed > 0);
    const int chunks = (a.V + r.shift + kVerifyChunk - 1) / kVerifyChunk;
    if (stale) {
      upto = verify_runs(sums, chunks);
      if (Z.hi > 0.f || a.q == nullptr) Z = from_lane(upto, 31);
    }
    if (!(Z.hi > 0.f) && removed > 0) {
      // nothing is left: the draft has as much everywhere.  The target's own
      // weights then, summed by this warp alone
      removed = 0;
      A = none;
      r.q = nullptr;
#pragma unroll 1
      for (int i = 0; i < chunks; ++i) {
        const Pair z = verify_chunk_alone(a, &s, r, i, 0);
        if (lane == 0) sums[i] = z;
      }
      __syncwarp();
      upto = verify_runs(sums, chunks);
      Z = from_lane(upto, 31);
    }
    if (Z.hi > 0.f && Z.hi < INFINITY)
      token = verify_draw(a, &s, sums, r, A, removed, upto, times(Pair{u, 0.f}, Z));
    bad = token < 0;
  }
  for (int i = count + lane; i < a.A; i += 32) a.accept_idx[static_cast<size_t>(b) * a.A + i] = -1;
  if (lane == 0) {
    a.accept_counts[b] = count;
    a.next_tokens[b] = token;
    if (bad) atomicOr(a.err, PKV_DEVERR_TREE);
  }
  if (done) cluster_wait();
}

cudaError_t launch_verify_tree(const VerifyArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = (a.V + 3 + kVerifyChunk - 1) / kVerifyChunk;
  // CTAs a sequence: up to four for each SM in all, and no more than have chunks
  int ranks = 1;
  while (ranks < kVerifyCluster && ranks * kVerifyWarps < chunks && 2 * ranks * static_cast<long long>(a.B) <= 4LL * num_sms) ranks *= 2;
  if (ranks > 8) {
    cudaError_t e = cudaFuncSetAttribute(verify_tree_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  const size_t smem = sizeof(Pair) * static_cast<size_t>(chunks);
  if (sizeof(VerifyShared) + smem > 48 * 1024) {  // (above 194,557 tokens: 380 chunk sums fit beside VerifyShared)
    cudaError_t e = cudaFuncSetAttribute(verify_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Pair) * kVerifyMaxChunks);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ranks);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_tree_kernel, a);
}

}  // namespace pkv
