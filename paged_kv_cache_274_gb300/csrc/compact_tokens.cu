// Accepted draft tokens moved together, in every cache slot.
//
// A verified draft of m nodes occupies positions base .. base + m - 1 of its
// sequence (base = n - m).  Of it the path idx[0] < idx[1] < ... is kept: the
// K and V rows of node idx[i] move to position base + i.  As idx[i] >= i, a
// row's new place never lies behind its old one, and no later row is read from
// a place that an earlier one was written to; so a thread that moves one
// 16-byte chunk of the rows in order, eight loads before their stores, needs
// no other ordering.
//
// One-byte pages: a row that moves to a page with the same parameters keeps
// its codes; else each code's value (code x scale, for INT8 (code - zero) x
// scale, in fp32) is quantised with the new page's parameters as an append
// does.
//
// One CTA per (sequence, cache slot) takes all KV heads of K and V.  Bound by
// latency, the chain of loads from the counts to the path, the table, the page
// parameters and the rows, which every CTA walks for itself: 32 bf16 slots of 64
// sequences with 1.7 moved rows each, 28.5 MB read and written (4.2 us at the
// copy rate; a pass after another finds them in L2), take 10 us (13 with a
// 64-bit division per row's offset); 8 E4M3 slots of 128 sequences with 1.9 rows,
// 8 MB (1.2 us), 10 us with the host's call, 8 to 10 us cold under a profile.
#include <algorithm>

#include "kv_append.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kCompactThreads = 256;
constexpr int kCompactBatch = 8;  // rows in flight per thread

template <int KV>
__device__ __forceinline__ uint4 requantise(uint4 x, const float* params, size_t src, size_t dst) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (KV == PKV_KV_FP8_E4M3) {
    const float s = __ldg(params + src), d = __ldg(params + dst);
    if (__float_as_uint(s) == __float_as_uint(d)) return x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2];
      e4m3x4_to_f16x2x2(w[i], h[0], h[1]);
      uint32_t o = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
        const float2 v = make_float2(__fdiv_rn(__fmul_rn(f.x, s), d), __fdiv_rn(__fmul_rn(f.y, s), d));
        o |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)) << (16 * k);
      }
      w[i] = o;
    }
  } else if constexpr (KV == PKV_KV_INT8) {
    const float2 s = __ldg(reinterpret_cast<const float2*>(params) + src);
    const float2 d = __ldg(reinterpret_cast<const float2*>(params) + dst);
    if (__float_as_uint(s.x) == __float_as_uint(d.x) && __float_as_uint(s.y) == __float_as_uint(d.y)) return x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t o = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float code = static_cast<float>(static_cast<int8_t>(w[i] >> (8 * k)));
        o |= int8_code(__fmul_rn(__fsub_rn(code, s.y), s.x), d.x, d.y) << (8 * k);
      }
      w[i] = o;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int KV>  // pkv_kv_dtype
__global__ void __launch_bounds__(kCompactThreads) compact_tokens_kernel(const CompactArgs a) {
  // per row: blocks (-1: stays where it is) and places in them
  __shared__ int s_src[PKV_MAX_QUERY_TOKENS], s_dst[PKV_MAX_QUERY_TOKENS];
  __shared__ uint16_t s_from[PKV_MAX_QUERY_TOKENS], s_to[PKV_MAX_QUERY_TOKENS];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / a.S, slot = blockIdx.x - b * a.S;
  const int n = a.context_lens[b], take = a.counts[b];
  const int nodes = a.node_counts != nullptr ? a.node_counts[b] : a.T;
  if (n == 0 && a.prev_lens != nullptr) {  // refused by extend_tables, or ended (block-uniform)
    if (slot == 0 && tid == 0) a.seq_lens[b] = a.new_lens[b] == -1 ? 0 : a.prev_lens[b];
    return;
  }
  const int base = n - nodes;
  unsigned err = 0;
  if (n < 0 || n > a.MB * a.bs) err |= PKV_DEVERR_CONTEXT_LEN;
  else if (nodes < 0 || nodes > a.T || take < 0 || take > min(a.A, nodes) || (take > 0 && base < 0)) err |= PKV_DEVERR_TREE;
  if (err == 0) {
    for (int i = tid; i < take; i += blockDim.x) {
      const int u = a.idx[static_cast<size_t>(b) * a.A + i];
      const int before = i > 0 ? a.idx[static_cast<size_t>(b) * a.A + i - 1] : -1;
      if (u <= before || u >= nodes) {
        err |= PKV_DEVERR_TREE;
      } else if (u != i) {
        const int ps = base + u, pd = base + i;
        const int js = ps / a.bs, jd = pd / a.bs;
        const int es = a.block_tables[static_cast<size_t>(b) * a.MB + js];
        const int ed = a.block_tables[static_cast<size_t>(b) * a.MB + jd];
        if (static_cast<unsigned>(es) >= static_cast<unsigned>(a.NB) || static_cast<unsigned>(ed) >= static_cast<unsigned>(a.NB))
          err |= PKV_DEVERR_BLOCK_ID;
        s_src[i] = es;
        s_dst[i] = ed;
        s_from[i] = static_cast<uint16_t>(ps - js * a.bs);
        s_to[i] = static_cast<uint16_t>(pd - jd * a.bs);
      } else {
        s_src[i] = -1;
      }
    }
  }
  // a sequence with anything wrong stays as it is (every thread learns of it)
  const bool wrong = __syncthreads_or(err != 0);
  if (slot == 0) {
    if (err) atomicOr(a.err, err);
    if (tid == 0) {
      const bool lens_ok = n >= 0 && n <= a.MB * a.bs && nodes >= 0 && nodes <= a.T;
      a.seq_lens[b] = !wrong && take > 0 ? base + take : (lens_ok ? max(base, 0) : 0);
    }
  }
  if (wrong || take == 0) return;
  int first = 0;  // leading rows that stay (idx[i] == i only up to the first that moves)
  while (first < take && s_src[first] < 0) ++first;
  constexpr int kElem = KV == PKV_KV_BF16 ? 2 : 1;
  const int row_chunks = a.D * kElem / 16;
  const int per_tensor = a.Hkv * row_chunks;
  for (int c = tid; c < 2 * per_tensor; c += blockDim.x) {
    const bool is_v = c >= per_tensor;
    const int r = is_v ? c - per_tensor : c;
    const int h = r / row_chunks, chunk = r - h * row_chunks;
    uint4* cache = reinterpret_cast<uint4*>(is_v ? a.vc : a.kc);
    const float* params = is_v ? a.vs : a.ks;
    const int64_t slot_pages = static_cast<int64_t>(slot) * a.NB;
    auto page_of = [&](int block) { return (slot_pages + block) * a.Hkv + h; };
    auto chunk_of = [&](int block, int token) { return (page_of(block) * a.bs + token) * row_chunks + chunk; };
    for (int i0 = first; i0 < take; i0 += kCompactBatch) {
      uint4 x[kCompactBatch];
#pragma unroll
      for (int k = 0; k < kCompactBatch; ++k)
        if (i0 + k < take) x[k] = cache[chunk_of(s_src[i0 + k], s_from[i0 + k])];
#pragma unroll
      for (int k = 0; k < kCompactBatch; ++k)
        if (i0 + k < take) {
          const int dst = s_dst[i0 + k];
          if constexpr (KV != PKV_KV_BF16) x[k] = requantise<KV>(x[k], params, page_of(s_src[i0 + k]), page_of(dst));
          cache[chunk_of(dst, s_to[i0 + k])] = x[k];
        }
    }
  }
}

cudaError_t launch_compact_tokens(int kv_dtype, const CompactArgs& a, cudaStream_t stream) {
  const int chunks = 2 * a.Hkv * a.D * (kv_dtype == PKV_KV_BF16 ? 2 : 1) / 16;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.S));
  cfg.blockDim = dim3(static_cast<unsigned>(std::min(kCompactThreads, (chunks + 31) / 32 * 32)));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = kv_dtype == PKV_KV_INT8        ? compact_tokens_kernel<PKV_KV_INT8>
                : kv_dtype == PKV_KV_FP8_E4M3 ? compact_tokens_kernel<PKV_KV_FP8_E4M3>
                                              : compact_tokens_kernel<PKV_KV_BF16>;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace pkv
