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
// but A, and a removed token's P is 0 by itself.
//
// The drawn token is a border among sums over the vocabulary, so everything is
// summed to 2^-44 or better: p - A q is kept as an unevaluated sum of two
// floats (error-free transformations of addition and product, T. J. Dekker and
// D. E. Knuth), so are the running sums; a chunk's sum is a double.  Doubles
// per element would be bound by the fp64 units (2 operations a clock and SM).
//
// What bounds it: the rows of the nodes where the walk loses a child or ends,
// from HBM, and for a small batch the chain of loads.  One cluster of up to 8
// CTAs per sequence.  Its first CTA walks (a warp; the nodes' own p and q are
// gathered beforehand, side by side) and tells the others by distributed shared
// memory which row to sum next; the CTAs take its chunks of 512 values in turn.
// Only the first CTA decides, so the others cannot come to another end.
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
constexpr int kVerifyCluster = 8;

// An unevaluated sum hi + lo.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ void add_to(Pair& x, const Pair& y) {
  const Pair s = two_sum(x.hi, y.hi);
  const float lo = __fadd_rn(s.lo, __fadd_rn(x.lo, y.lo));
  x.hi = __fadd_rn(s.hi, lo);
  x.lo = __fsub_rn(lo, __fsub_rn(x.hi, s.hi));
}
// What is negative or not finite counts as 0.
__device__ __forceinline__ Pair weight(float p) { return {p > 0.f && p < INFINITY ? p : 0.f, 0.f}; }
// max(p - (ah + al) q, 0), likewise.
__device__ __forceinline__ Pair weight_left(float p, float q, float ah, float al) {
  const float h = __fmul_rn(ah, q);
  const float l = fmaf(al, q, fmaf(ah, q, -h));
  const Pair d = two_sum(p, -h);
  const float lo = __fsub_rn(d.lo, l);
  const bool some = __fadd_rn(d.hi, lo) > 0.f;
  return {some ? d.hi : 0.f, some ? lo : 0.f};
}
__device__ __forceinline__ double value(const Pair& x) { return static_cast<double>(x.hi) + static_cast<double>(x.lo); }
__device__ __forceinline__ Pair warp_total(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair y{__shfl_xor_sync(kFull, x.hi, o), __shfl_xor_sync(kFull, x.lo, o)};
    add_to(x, y);
  }
  return x;
}

struct VerifyShared {
  // what to sum next, written by the cluster's first CTA
  int row;       // of the sequence; -1: nothing more
  int removed;   // tokens in `gone`
  int want_y;
  float ah, al;
  double y_part[kVerifyCluster * kVerifyWarps];  // (first CTA)
  int gone[PKV_MAX_QUERY_TOKENS];                // tokens of the rejected children
  // the nodes (first CTA)
  int token[PKV_MAX_QUERY_TOKENS], parent[PKV_MAX_QUERY_TOKENS];
  float r[PKV_MAX_QUERY_TOKENS], p[PKV_MAX_QUERY_TOKENS], q[PKV_MAX_QUERY_TOKENS];
};

// 512 values of a row from e0 on, 16 a lane: lane's value k is at
// e0 + verify_at(k, lane); 0 past the row.
template <bool VEC>
__device__ __forceinline__ int verify_at(int k, int lane) {
  return VEC ? (k / 4) * 128 + lane * 4 + k % 4 : k * 32 + lane;
}
template <bool VEC>
__device__ __forceinline__ void verify_load(float (&x)[kPer], const float* row, int e0, int V, int lane) {
  if constexpr (VEC) {  // (V is a multiple of 4)
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
      const int e = e0 + verify_at<true>(4 * k, lane);
      const float4 v = e < V ? __ldg(reinterpret_cast<const float4*>(row + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[4 * k] = v.x;
      x[4 * k + 1] = v.y;
      x[4 * k + 2] = v.z;
      x[4 * k + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = e0 + verify_at<false>(k, lane);
      x[k] = e < V ? __ldg(row + e) : 0.f;
    }
  }
}

// This CTA's chunks of the row: sums of max(p - A q, 0) to the first CTA's
// `sums`, this warp's sum of the Q that are left to its y_part.
template <bool VEC, bool DRAFT>
__device__ __forceinline__ void verify_pass(const VerifyArgs& a, const VerifyShared* s, double* sums0, double* y_part0, const float* p,
                                            const float* q, int chunks, int rank, int ranks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float ah = s->ah, al = s->al;
  const int removed = s->removed;
  const bool want_y = s->want_y != 0;
  Pair y{0.f, 0.f};
#pragma unroll 1
  for (int i = warp * ranks + rank; i < chunks; i += kVerifyWarps * ranks) {
    const int e0 = i * kVerifyChunk;
    float pv[kPer], qv[kPer];
    verify_load<VEC>(pv, p, e0, a.V, lane);
    if constexpr (DRAFT) verify_load<VEC>(qv, q, e0, a.V, lane);
    Pair z{0.f, 0.f};
    auto drop = [&](float (&x)[kPer]) {  // rejected children's tokens
#pragma unroll 1
      for (int g = 0; g < removed; ++g) {
        const int d = s->gone[g] - e0;
        if (static_cast<unsigned>(d) < static_cast<unsigned>(kVerifyChunk)) {
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if (verify_at<VEC>(k, lane) == d) x[k] = 0.f;
        }
      }
    };
    if constexpr (!DRAFT) drop(pv);
#pragma unroll
    for (int k = 0; k < kPer; ++k) add_to(z, DRAFT ? weight_left(pv[k], qv[k], ah, al) : weight(pv[k]));
    if constexpr (DRAFT) {
      if (want_y) {
        drop(qv);
#pragma unroll
        for (int k = 0; k < kPer; ++k) add_to(y, Pair{qv[k], 0.f});
      }
    }
    z = warp_total(z);
    if (lane == 0) sums0[i] = value(z);
  }
  if (want_y) {
    y = warp_total(y);
    if (lane == 0) y_part0[rank * kVerifyWarps + warp] = value(y);
  }
}

// Inclusive scan over the warp.
__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// The first index whose partial sum exceeds u times the whole (the last with
// any weight, should rounding leave none).  One warp.
__device__ __forceinline__ int verify_draw(const VerifyArgs& a, const VerifyShared* s, const double* sums, int chunks, const float* p,
                                           const float* q, float ah, float al, int removed, double target) {
  const int lane = threadIdx.x & 31;
  // chunk by chunk, a run of chunks per lane
  const int per = (chunks + 31) / 32, c0 = min(lane * per, chunks), c1 = min(c0 + per, chunks);
  double mine = 0.0;
  for (int i = c0; i < c1; ++i) mine += sums[i];
  const double upto = warp_scan(mine, lane);
  double before = upto - mine;
  int chunk = -1, any = -1;
  double base = 0.0;
  for (int i = c0; i < c1; ++i) {
    if (sums[i] > 0.0) {
      any = i;
      if (chunk < 0 && before + sums[i] > target) {
        chunk = i;
        base = before;
      }
    }
    before += sums[i];
  }
  const unsigned found = __ballot_sync(kFull, chunk >= 0), some = __ballot_sync(kFull, any >= 0);
  if (some == 0) return -1;
  const bool last = found == 0;
  const int from = last ? 31 - __clz(some) : __ffs(found) - 1;
  chunk = __shfl_sync(kFull, last ? any : chunk, from);
  base = __shfl_sync(kFull, base, from);
  // 16 values a lane in their order
  const int e0 = chunk * kVerifyChunk + lane * kPer;
  double w[kPer], sum = 0.0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int e = e0 + k;
    Pair x{0.f, 0.f};
    if (e < a.V) {
      const float pv = __ldg(p + e);
      x = q != nullptr ? weight_left(pv, __ldg(q + e), ah, al) : weight(pv);
    }
    w[k] = value(x);
  }
  if (q == nullptr) {
    for (int g = 0; g < removed; ++g) {
      const int d = s->gone[g] - e0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (k == d) w[k] = 0.0;
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum += w[k];
  double at = base + (warp_scan(sum, lane) - sum);
  int hit = -1, tail = -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    at += w[k];
    if (w[k] > 0.0) {
      tail = e0 + k;
      if (hit < 0 && at > target) hit = e0 + k;
    }
  }
  const unsigned hits = last ? 0u : __ballot_sync(kFull, hit >= 0), tails = __ballot_sync(kFull, tail >= 0);
  if (hits != 0) return __shfl_sync(kFull, hit, __ffs(hits) - 1);
  return tails != 0 ? __shfl_sync(kFull, tail, 31 - __clz(tails)) : -1;
}

__global__ void __launch_bounds__(kVerifyThreads) verify_tree_kernel(const VerifyArgs a) {
  __shared__ VerifyShared s;
  extern __shared__ double sums[];  // (first CTA) of the chunks
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (a.V + kVerifyChunk - 1) / kVerifyChunk;
  pdl_trigger();
  pdl_wait();
  const size_t seq = static_cast<size_t>(b) * a.T;
  auto row_p = [&](int t) { return a.p + (seq + t) * a.p_stride; };
  auto row_q = [&](int t) { return a.q + (seq + t) * a.q_stride; };

  // the nodes, and what the target and the draft give them
  int nodes = 0;
  bool bad = false;
  if (rank == 0) {
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
  double A = 0.0, Z = 1.0, Y = 1.0;
  bool summed = false;    // `sums` are those of P as it is
  bool walking = nodes > 0, whole = false;
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
  auto tell = [&](int row, bool want_y) {
    const float ah = static_cast<float>(A), al = static_cast<float>(A - static_cast<double>(ah));
    if (lane < ranks) {
      VerifyShared* to = cluster.map_shared_rank(&s, lane);
      to->row = row;
      to->removed = removed;
      to->want_y = want_y ? 1 : 0;
      to->ah = ah;
      to->al = al;
      if (removed > 0) to->gone[removed - 1] = s.token[next - 1];
    }
  };
  double* sums0 = cluster.map_shared_rank(sums, 0);
  double* y_part0 = cluster.map_shared_rank(s.y_part, 0);

  cluster.sync();  // every CTA of the cluster runs
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
        const double q = was ? 0.0 : static_cast<double>(s.q[c]);
        double left = static_cast<double>(s.p[c]) - (a.q != nullptr ? A * static_cast<double>(s.q[c]) : 0.0);
        if (!(left > 0.0) || (a.q == nullptr && was)) left = 0.0;
        if (static_cast<double>(s.r[c]) * (a.q != nullptr ? q : 1.0) * Z < left * Y) {
          if (lane == 0) a.accept_idx[static_cast<size_t>(b) * a.A + count] = c;
          ++count;
          at = c;
          removed = 0;
          A = 0.0;
          Z = Y = 1.0;
          summed = false;
        } else {
          A += Y > 0.0 ? Z / Y : 0.0;
          ++removed;
          tell(at, a.q != nullptr && child(next) >= 0);
          ask = true;
        }
      }
      if (!ask && nodes > 0) {
        if (!summed) {  // the target's own weights
          tell(at, false);
          ask = true;
        } else if (!(Z > 0.0) && !whole) {
          // nothing is left: the draft has as much everywhere
          whole = true;
          removed = 0;
          A = 0.0;
          tell(at, false);
          ask = true;
        }
      }
      if (!ask) tell(-1, false);
      summed = true;
    }
    cluster.sync();  // the request is there
    const int row = s.row;
    if (row < 0) break;
    const float* p = row_p(row);
    const float* q = a.q != nullptr ? row_q(row) : nullptr;
    // (one test for all rows: strides and bases of 16 bytes)
    if (a.q != nullptr)
      a.vec ? verify_pass<true, true>(a, &s, sums0, y_part0, p, q, chunks, rank, ranks)
            : verify_pass<false, true>(a, &s, sums0, y_part0, p, q, chunks, rank, ranks);
    else
      a.vec ? verify_pass<true, false>(a, &s, sums0, y_part0, p, q, chunks, rank, ranks)
            : verify_pass<false, false>(a, &s, sums0, y_part0, p, q, chunks, rank, ranks);
    cluster.sync();  // the sums are there
    if (rank == 0 && warp == 0) {
      double z = 0.0, y = 0.0;
      for (int i = lane; i < chunks; i += 32) z += sums[i];
      Z = warp_sum(z);
      if (a.q != nullptr && s.want_y) {
        for (int i = lane; i < ranks * kVerifyWarps; i += 32) y += s.y_part[i];
        Y = warp_sum(y);
      } else {
        Y = 1.0;
      }
    }
  }
  if (rank != 0 || warp != 0) return;
  if (nodes > 0) {
    const bool finite = Z > 0.0 && Z < INFINITY;
    if (finite) {
      const float ah = static_cast<float>(A), al = static_cast<float>(A - static_cast<double>(ah));
      token = verify_draw(a, &s, sums, chunks, row_p(at), a.q != nullptr ? row_q(at) : nullptr, ah, al, removed,
                          static_cast<double>(a.sample_uniforms[b]) * Z);
    }
    bad = token < 0;
  }
  for (int i = count + lane; i < a.A; i += 32) a.accept_idx[static_cast<size_t>(b) * a.A + i] = -1;
  if (lane == 0) {
    a.accept_counts[b] = count;
    a.next_tokens[b] = token;
    if (bad) atomicOr(a.err, PKV_DEVERR_TREE);
  }
}

cudaError_t launch_verify_tree(const VerifyArgs& a, int num_sms, cudaStream_t stream) {
  const int chunks = (a.V + kVerifyChunk - 1) / kVerifyChunk;
  // CTAs a sequence: two for each SM in all, and no more than have chunks
  int ranks = 1;
  while (ranks < kVerifyCluster && ranks * kVerifyWarps < chunks && 2 * ranks * static_cast<long long>(a.B) <= 4LL * num_sms) ranks *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ranks);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = sizeof(double) * static_cast<size_t>(chunks);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_tree_kernel, a);
}

}  // namespace pkv
