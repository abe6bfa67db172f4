// Norms of each head of the queries and keys, their rotation by the tokens'
// positions, and the append of keys and values, in one pass.
//
// Of a head's row x of D values (fp32 throughout, one rounding at the end):
//   y = x / sqrt(mean(x^2) + eps) * w          (w the norm's weights; optional)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   for each pair i
// with the angle positions[axis(i)] * inv_freq[i].
//
// A row takes D / 8 lanes, so a warp has two (D 128) or four rows at a time.  A
// lane holds four pairs, two runs of four values: both elements of its pairs, so
// the rotation needs no exchange (with 16 consecutive bytes a lane, the halves'
// partners came by four shuffles and eight more conversions a row group).  What
// depends on the token alone is made once per warp: the row's factor r times
// x_a (w_a cos) - x_b (w_b sin), and likewise for b.
//
// Angles are kept in turns: the host gives each frequency as a fraction of a
// turn per position in 2^-64, to two units (rope_turns.h), and position x
// frequency modulo 2^64 is an integer product: 2^-31 of half a turn at the last
// int32 position.  The nearest quarter turn comes off as an integer too, and the
// rest, at most an eighth of a turn, goes to sincospif as a float, off by up to
// 2^-27: an angle is off by less than 2^-26 of half a turn wherever the token is.
// (With the whole turn as one float, 2^-24, E4M3 keys took the other neighbour
// twice as often.)
//
// What bounds it: HBM for long prompts, the call on the host for a decode step;
// see the times at launch_rope_append.
#include <algorithm>

#include "kv_append.cuh"

namespace pkv {

constexpr int kRopeThreads = 128;
constexpr int kRopeBatch = 4;  // row groups whose loads are in flight together
constexpr int kRopePair = 2;   // and are turned together
constexpr int kRopeCtas = 8;   // of an SM

// A lane's values: x[0..3] the first run, x[4..7] the second.  Pair k is x[k],
// x[k + 4] (halves) or x[2 k], x[2 k + 1] (neighbours).
template <bool HALVES>
__device__ __forceinline__ constexpr int rope_first(int k) {
  return HALVES ? k : 2 * k;
}
template <bool HALVES>
__device__ __forceinline__ constexpr int rope_second(int k) {
  return HALVES ? k + 4 : 2 * k + 1;
}

__device__ __forceinline__ void unpack8(float (&x)[8], const uint2& a, const uint2& b) {
  x[0] = bf16lo_to_f32(a.x);
  x[1] = bf16hi_to_f32(a.x);
  x[2] = bf16lo_to_f32(a.y);
  x[3] = bf16hi_to_f32(a.y);
  x[4] = bf16lo_to_f32(b.x);
  x[5] = bf16hi_to_f32(b.x);
  x[6] = bf16lo_to_f32(b.y);
  x[7] = bf16hi_to_f32(b.y);
}

// The norm and the rotation of two row groups, so that the norms' chains of
// shuffles run side by side.  w: the lane's weights (bf16), cs, sn of its pairs.
template <int D, bool HALVES>
__device__ __forceinline__ void turn_rows(float (&y)[kRopePair][8], const uint2& w0, const uint2& w1, const float (&cs)[4], const float (&sn)[4],
                                          bool norm, float eps, bool turned) {
  constexpr int kLanes = D / 8;
  if (norm) {
    float r[kRopePair];
#pragma unroll
    for (int u = 0; u < kRopePair; ++u) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j += 2) ffma2(s0, s1, y[u][j], y[u][j + 1], y[u][j], y[u][j + 1], s0, s1);
      r[u] = s0 + s1;
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < kRopePair; ++u) r[u] += __shfl_xor_sync(kFull, r[u], o);
    float w[8];
    unpack8(w, w0, w1);
#pragma unroll
    for (int u = 0; u < kRopePair; ++u) {
      r[u] = rsqrtf(fmaf(r[u], 1.f / D, eps));
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        fmul2(y[u][j], y[u][j + 1], y[u][j], y[u][j + 1], r[u], r[u]);
        fmul2(y[u][j], y[u][j + 1], y[u][j], y[u][j + 1], w[j], w[j + 1]);
      }
    }
  }
  if (turned) {
#pragma unroll
    for (int u = 0; u < kRopePair; ++u) {
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        float& a0 = y[u][rope_first<HALVES>(k)];
        float& a1 = y[u][rope_first<HALVES>(k + 1)];
        float& b0 = y[u][rope_second<HALVES>(k)];
        float& b1 = y[u][rope_second<HALVES>(k + 1)];
        float t0, t1, v0, v1;
        if constexpr (HALVES) {  // (two pairs to a register pair)
          fmul2(t0, t1, b0, b1, -sn[k], -sn[k + 1]);
          fmul2(v0, v1, a0, a1, sn[k], sn[k + 1]);
          ffma2(a0, a1, a0, a1, cs[k], cs[k + 1], t0, t1);
          ffma2(b0, b1, b0, b1, cs[k], cs[k + 1], v0, v1);
        } else {
          t0 = b0 * sn[k];
          t1 = b1 * sn[k + 1];
          v0 = a0 * sn[k];
          v1 = a1 * sn[k + 1];
          a0 = fmaf(a0, cs[k], -t0);
          a1 = fmaf(a1, cs[k + 1], -t1);
          b0 = fmaf(b0, cs[k], v0);
          b1 = fmaf(b1, cs[k + 1], v1);
        }
      }
    }
  }
}

template <int D, int KV, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kHeads = kRopeBatch * kRows;  // heads of a batch
  __shared__ uint64_t freq[64];
  __shared__ int axis[64];
  pdl_trigger();
  // (once per CTA: lanes that read constants apart take a turn each)
  if (threadIdx.x < a.R / 2) {
    freq[threadIdx.x] = a.turns[threadIdx.x];
    axis[threadIdx.x] = a.axis[threadIdx.x];
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
  // the lane's runs of four values; lanes past the rotated part have eight in a row
  const bool turned = 8 * c < a.R;
  const int e0 = HALVES && turned ? 4 * c : 8 * c, e1 = HALVES && turned ? a.R / 2 + 4 * c : 8 * c + 4;
  const int nq = (a.Hq + kHeads - 1) / kHeads, nk = a.k_new ? (a.app.Hkv + kHeads - 1) / kHeads : 0;  // batches
  const int batches = nq + 2 * nk, per = (batches + a.parts - 1) / a.parts;
  pdl_wait();
  const unsigned items = static_cast<unsigned>(a.app.N) * a.parts;  // (less than 2^31, as the host sees to)
#pragma unroll 1
  for (unsigned item = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); item < items; item += gridDim.x * (kRopeThreads / 32)) {
    const unsigned token = item / a.parts;
    const int begin = static_cast<int>(item - token * a.parts) * per, end = min(batches, begin + per);
    long long slot = 0;
    if (a.app.slot_mapping != nullptr) {
      slot = __ldg(a.app.slot_mapping + token);
      if (slot < 0 || slot >= a.app.nslots) {
        if (slot != -1 && begin == 0 && lane == 0) atomicOr(a.app.err, PKV_DEVERR_SLOT);
        continue;
      }
    }
    float cs[4], sn[4];  // of the lane's pairs: angles 4 c .. 4 c + 3
    {
      float cs2[2] = {1.f, 1.f}, sn2[2] = {0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 2; ++s) {  // lane t makes the angles 2 t and 2 t + 1
        const int i = 2 * lane + s;
        if (i < a.R / 2) {
          const long long pos = __ldg(a.positions + static_cast<size_t>(axis[i]) * a.app.N + token);
          const uint64_t turn = static_cast<uint64_t>(pos) * freq[i], quarter = (turn + (1ull << 61)) >> 62;
          float sn, cs;
          sincospif(static_cast<float>(static_cast<int64_t>(turn - (quarter << 62))) * 0x1p-63f, &sn, &cs);
          if (quarter & 1) {
            const float was = sn;
            sn = cs;
            cs = -was;
          }
          sn2[s] = (quarter & 2) ? -sn : sn;
          cs2[s] = (quarter & 2) ? -cs : cs;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        cs[k] = __shfl_sync(kFull, cs2[k & 1], 2 * c + k / 2);
        sn[k] = __shfl_sync(kFull, sn2[k & 1], 2 * c + k / 2);
      }
    }
    const int shift = a.app.bs == 32 ? 5 : 4;  // (blocks of 16 or 32 tokens)
    const int blk = static_cast<int>(slot >> shift), off = static_cast<int>(slot) & (a.app.bs - 1);

    // batches lo .. hi - 1 of the queries' (0), keys' (1) or values' (2) rows
    auto rows = [&](auto tag, int lo, int hi) {
      constexpr int which = decltype(tag)::value;
      const int heads = which == 0 ? a.Hq : a.app.Hkv;
      const __nv_bfloat16* src = which == 0 ? a.q + token * a.q_stride : which == 1 ? a.k + token * a.k_stride : a.v + token * a.v_stride;
      const uint16_t* weight = which == 0 ? a.qw : which == 1 ? a.kw : nullptr;
      uint2 w0 = make_uint2(0, 0), w1 = w0;
      if (weight != nullptr) {
        w0 = __ldg(reinterpret_cast<const uint2*>(weight + e0));
        w1 = __ldg(reinterpret_cast<const uint2*>(weight + e1));
      }
      // where head 0's row goes, and how far apart the heads' rows are there
      constexpr int elem = which == 0 || KV == PKV_KV_BF16 ? 2 : 1;
      uint8_t* dst;
      int apart;
      [[maybe_unused]] const float* scales = nullptr;
      if constexpr (which == 0) {
        dst = reinterpret_cast<uint8_t*>(a.q_out + token * a.out_stride);
        apart = D * elem;
      } else {
        const long long page = static_cast<long long>(blk) * a.app.Hkv;
        dst = (which == 1 ? a.app.kc : a.app.vc) + (page * a.app.bs + off) * (D * elem);
        apart = a.app.bs * (D * elem);
        if constexpr (KV != PKV_KV_BF16) scales = (which == 1 ? a.app.ks : a.app.vs) + page * (KV == PKV_KV_INT8 ? 2 : 1);
      }
#pragma unroll 1
      for (int i = lo; i < hi; ++i) {
        const int h0 = i * kHeads + sub;
        const __nv_bfloat16* from = src + h0 * D;
        uint8_t* out = dst + static_cast<long long>(h0) * apart;
        uint2 xa[kRopeBatch], xb[kRopeBatch];
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
          const int h = h0 + u * kRows;
          xa[u] = xb[u] = make_uint2(0, 0);
          if (h < heads) {
            xa[u] = __ldcs(reinterpret_cast<const uint2*>(from + u * kRows * D + e0));
            xb[u] = __ldcs(reinterpret_cast<const uint2*>(from + u * kRows * D + e1));
          }
        }
#pragma unroll
        for (int u = 0; u < kRopeBatch; u += kRopePair) {
          float y[kRopePair][8];
          if constexpr (which < 2 || elem == 1) {
#pragma unroll
            for (int v = 0; v < kRopePair; ++v) unpack8(y[v], xa[u + v], xb[u + v]);
          }
          if constexpr (which < 2) turn_rows<D, HALVES>(y, w0, w1, cs, sn, weight != nullptr, a.eps, turned);
#pragma unroll
          for (int v = 0; v < kRopePair; ++v) {
            const int h = h0 + (u + v) * kRows;
            if (h >= heads) continue;
            uint8_t* to = out + (u + v) * kRows * apart;
            if constexpr (elem == 2) {
              // (values keep their bits, NaNs too)
              *reinterpret_cast<uint2*>(to + 2 * e0) =
                  which == 2 ? xa[u + v] : make_uint2(pack_bf16x2(y[v][0], y[v][1]), pack_bf16x2(y[v][2], y[v][3]));
              *reinterpret_cast<uint2*>(to + 2 * e1) =
                  which == 2 ? xb[u + v] : make_uint2(pack_bf16x2(y[v][4], y[v][5]), pack_bf16x2(y[v][6], y[v][7]));
            } else {
              uint32_t w[2] = {0u, 0u};
              if constexpr (KV == PKV_KV_INT8) {
                const float2 sz = __ldg(reinterpret_cast<const float2*>(scales) + h);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j >> 2] |= int8_code(y[v][j], sz.x, sz.y) << (8 * (j & 3));
              } else {
                const float scale = __ldg(scales + h);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                                   make_float2(__fdiv_rn(y[v][2 * j], scale), __fdiv_rn(y[v][2 * j + 1], scale)), __NV_SATFINITE, __NV_E4M3))
                               << (16 * (j & 1));
              }
              *reinterpret_cast<uint32_t*>(to + e0) = w[0];
              *reinterpret_cast<uint32_t*>(to + e1) = w[1];
            }
          }
        }
      }
    };
    auto span = [&](auto tag, int base, int n) {
      const int lo = max(begin - base, 0), hi = min(end - base, n);
      if (lo < hi) rows(tag, lo, hi);
    };
    span(std::integral_constant<int, 0>{}, 0, nq);
    span(std::integral_constant<int, 1>{}, nq, nk);
    span(std::integral_constant<int, 2>{}, nq + nk, nk);
  }
}

template <int D, int KV>
static cudaError_t launch_rope(const RopeArgs& a, bool halves, const cudaLaunchConfig_t& cfg) {
  return halves ? cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KV, true>, a) : cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KV, false>, a);
}

// 8,192 tokens, 32 + 2 x 8 heads of 128 with norms, bf16 (202 MB): 36 us, 0.84 of
// the copy rate; 5,003 tokens, 64 + 2 x 8 heads, half of each turned, E4M3 cache
// (195 MB): 38 us, 0.78.  64 tokens (1.6 MB): 2.9 us in a graph, 5.8 a call, of
// which 5.3 are the host's.  A part of a token is two batches, so that its angles
// serve 16 rows or more (head_dim 64: 32); in us for these three: half the batches
// 36, 38, 5.8; one part 38, 47, 6.1; a batch a part 40, 41, 5.9.  The other forms of
// the first: head_dim 64 (101 MB) 20.9 us, 0.72, with 64 heads (168 MB) 32.0, 0.79;
// E4M3 cache (185 MB) 39 us, 0.71; INT8 (185 MB) 47 us, 0.59.  Tokens are cut
// into more parts only where that leaves warps idle.  (6 CTAs an SM: 37 and 38; 12:
// 55 and 45, with registers spilt.)
cudaError_t launch_rope_append(int kv_dtype, int D, bool halves, RopeArgs a, int num_sms, cudaStream_t stream) {
  const int heads = kRopeBatch * (32 / (D / 8));
  const int batches = (a.Hq + heads - 1) / heads + (a.k_new ? 2 * ((a.app.Hkv + heads - 1) / heads) : 0);
  const long long warps = static_cast<long long>(num_sms) * kRopeCtas * (kRopeThreads / 32);
  int parts = (batches + 1) / 2;
  if (static_cast<long long>(a.app.N) * parts < warps)
    parts = static_cast<int>(std::min<long long>(batches, (warps + a.app.N - 1) / a.app.N));
  a.parts = parts;
  const long long items = static_cast<long long>(a.app.N) * parts;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((std::min(items, warps) + kRopeThreads / 32 - 1) / (kRopeThreads / 32)));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kv_dtype == PKV_KV_INT8) return launch_rope<128, PKV_KV_INT8>(a, halves, cfg);
  if (kv_dtype == PKV_KV_FP8_E4M3) return launch_rope<128, PKV_KV_FP8_E4M3>(a, halves, cfg);
  return D == 64 ? launch_rope<64, PKV_KV_BF16>(a, halves, cfg) : launch_rope<128, PKV_KV_BF16>(a, halves, cfg);
}

}  // namespace pkv
