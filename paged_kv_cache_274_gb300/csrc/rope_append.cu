// Norms of each head of the queries and keys, their rotation by the tokens'
// positions, and the append of keys and values, in one pass.
//
// Of a head's row x of D values (fp32 throughout, one rounding at the end):
//   y = x / sqrt(mean(x^2) + eps) * w          (w the norm's weights; optional)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   for each pair i
// with the angle positions[axis(i)] * inv_freq[i].
//
// A row takes D / 8 lanes, 16 bytes each, so a warp loads two (D 128) or four
// rows at a time.  What depends on the token alone is made once per warp:
// out_j = r (x_j A_j + x_p B_j), where r is the row's norm factor, x_p the
// pair's other element, A = w_j cos and B = -/+ w_p sin.  A pair's elements lie
// in one lane (neighbours) or R / 16 lanes apart (halves; four shuffles of raw
// bf16 words).
//
// Angles are kept in turns: the host gives each frequency as a fraction of a
// turn per position in 2^-64, and position x frequency modulo 2^64 is an
// integer product, exact at any position.  Its upper 32 bits go to sincospif,
// so an angle is off by less than 2^-24 of half a turn wherever the token is.
//
// What bounds it: every row is read and written once; see the times at
// launch_rope_append.
#include <algorithm>

#include "kv_append.cuh"

namespace pkv {

constexpr int kRopeThreads = 128;
constexpr int kRopeBatch = 4;  // row groups whose loads are in flight together

// Coefficients of one tensor's rows in this lane: out = r (x a + x_p b).
struct RopeCoef {
  float a[8], b[8];
};

template <int D, bool HALVES>
__device__ __forceinline__ void rope_coef(RopeCoef& f, const uint16_t* weight, int c, int partner, bool turned, const float (&cs)[8],
                                          const float (&sn)[8]) {
  uint4 w = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), v = w;  // ones
  if (weight != nullptr) {
    w = __ldg(reinterpret_cast<const uint4*>(weight) + c);
    if (HALVES) v = __ldg(reinterpret_cast<const uint4*>(weight) + partner);
  }
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    auto at = [&](const uint32_t (&t)[4], int k) { return (k & 1) ? bf16hi_to_f32(t[k >> 1]) : bf16lo_to_f32(t[k >> 1]); };
    f.a[j] = at(ww, j) * (turned ? cs[j] : 1.f);
    f.b[j] = turned ? (HALVES ? at(vw, j) : at(ww, j ^ 1)) * sn[j] : 0.f;
  }
}

template <int D, int KV, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
  const long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const long long token = item / a.parts;
  if (token >= a.app.N) return;
  const int part = static_cast<int>(item - token * a.parts);
  long long slot = 0;
  if (a.app.slot_mapping != nullptr) {
    slot = __ldg(a.app.slot_mapping + token);
    if (slot < 0 || slot >= a.app.nslots) {
      if (slot != -1 && part == 0 && lane == 0) atomicOr(a.app.err, PKV_DEVERR_SLOT);
      return;
    }
  }
  // lane t: angles 2 t and 2 t + 1
  float cs2[2] = {1.f, 1.f}, sn2[2] = {0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int i = 2 * lane + s;
    if (i < a.R / 2) {
      const long long pos = __ldg(a.positions + static_cast<size_t>(a.axis[i]) * a.app.N + token);
      const uint64_t turn = static_cast<uint64_t>(pos) * a.turns[i];
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn2[s], &cs2[s]);
    }
  }
  const int half = a.R / 16;  // lanes of a half of the rotated part
  const bool turned = 8 * c < a.R, second = HALVES && c >= half;
  const int partner = !HALVES || !turned ? c : second ? c - half : c + half;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // halves: angles 8 (c mod half) + j; neighbours: 4 c + j / 2
    const int from = HALVES ? 4 * (second ? c - half : c) + j / 2 : 2 * c + j / 4;
    const int k = HALVES ? j & 1 : (j >> 1) & 1;
    cs[j] = __shfl_sync(kFull, cs2[k], from);
    const float s = __shfl_sync(kFull, sn2[k], from);
    sn[j] = (HALVES ? second : (j & 1) != 0) ? s : -s;
  }
  const int gq = (a.Hq + kRows - 1) / kRows, gk = a.k_new ? (a.app.Hkv + kRows - 1) / kRows : 0;
  const int groups = gq + 2 * gk, per = (groups + a.parts - 1) / a.parts;
  const int g_end = min(groups, (part + 1) * per);
  const long long blk = slot / a.app.bs;
  const int off = static_cast<int>(slot - blk * a.app.bs);

  // rows of q (which 0), k (1) or v (2): groups g0 .. g1 - 1 of that tensor
  auto rows = [&](auto which_tag, int g0, int g1) {
    constexpr int which = decltype(which_tag)::value;
    const int heads = which == 0 ? a.Hq : a.app.Hkv;
    const uint4* src = reinterpret_cast<const uint4*>((which == 0 ? a.q + token * a.q_stride : which == 1 ? a.k + token * a.k_stride : a.v + token * a.v_stride));
    RopeCoef f;
    bool norm = false;
    if constexpr (which < 2) {
      const uint16_t* w = which == 0 ? a.qw : a.kw;
      norm = w != nullptr;
      rope_coef<D, HALVES>(f, w, c, partner, turned, cs, sn);
    }
#pragma unroll 1
    for (int g = g0; g < g1; g += kRopeBatch) {
      uint4 x[kRopeBatch];
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        const int h = (g + u) * kRows + sub;
        x[u] = g + u < g1 && h < heads ? __ldcs(src + h * kLanes + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        const int h = (g + u) * kRows + sub;
        const bool live = g + u < g1 && h < heads;
        const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        float y[8] = {};
        if constexpr (which < 2) {
          float xf[8], r = 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xf[2 * j] = bf16lo_to_f32(xw[j]);
            xf[2 * j + 1] = bf16hi_to_f32(xw[j]);
          }
          if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(xf[j], xf[j], ss);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
          }
          float p[8];
          if constexpr (HALVES) {
            const int from = (lane & ~(kLanes - 1)) | partner;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w = __shfl_sync(kFull, xw[j], from);
              if (!turned) w = 0u;  // (an infinity times b = 0 would be NaN)
              p[2 * j] = bf16lo_to_f32(w);
              p[2 * j + 1] = bf16hi_to_f32(w);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = turned ? xf[j ^ 1] : 0.f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = r * fmaf(xf[j], f.a[j], p[j] * f.b[j]);
        }
        if (!live) continue;
        if constexpr (which == 0) {
          uint4* dst = reinterpret_cast<uint4*>(a.q_out + token * a.out_stride) + h * kLanes + c;
          *dst = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        } else {
          const long long page = blk * a.app.Hkv + h;
          const long long elem = (page * a.app.bs + off) * D + 8 * c;
          uint8_t* cache = which == 1 ? a.app.kc : a.app.vc;
          [[maybe_unused]] const float* scales = which == 1 ? a.app.ks : a.app.vs;
          if constexpr (which == 2 && KV != PKV_KV_BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[2 * j] = bf16lo_to_f32(xw[j]);
              y[2 * j + 1] = bf16hi_to_f32(xw[j]);
            }
          }
          if constexpr (KV == PKV_KV_BF16) {
            *reinterpret_cast<uint4*>(cache + 2 * elem) =
                which == 2 ? x[u]
                           : make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
          } else {
            uint32_t w[2] = {0u, 0u};
            if constexpr (KV == PKV_KV_INT8) {
              const float2 sz = __ldg(reinterpret_cast<const float2*>(scales) + page);
#pragma unroll
              for (int j = 0; j < 8; ++j) w[j >> 2] |= int8_code(y[j], sz.x, sz.y) << (8 * (j & 3));
            } else {
              const float scale = __ldg(scales + page);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[2 * j], scale), __fdiv_rn(y[2 * j + 1], scale)),
                                                                            __NV_SATFINITE, __NV_E4M3))
                             << (16 * (j & 1));
            }
            *reinterpret_cast<uint2*>(cache + elem) = make_uint2(w[0], w[1]);
          }
        }
      }
    }
  };
  const int g_begin = part * per;
  auto span = [&](auto tag, int base, int n) {
    const int lo = max(g_begin - base, 0), hi = min(g_end - base, n);
    if (lo < hi) rows(tag, lo, hi);
  };
  span(std::integral_constant<int, 0>{}, 0, gq);
  span(std::integral_constant<int, 1>{}, gq, gk);
  span(std::integral_constant<int, 2>{}, gq + gk, gk);
}

template <int D, int KV>
static cudaError_t launch_rope(const RopeArgs& a, bool halves, const cudaLaunchConfig_t& cfg) {
  return halves ? cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KV, true>, a) : cudaLaunchKernelEx(&cfg, rope_append_kernel<D, KV, false>, a);
}

cudaError_t launch_rope_append(int kv_dtype, int D, bool halves, RopeArgs a, int num_sms, cudaStream_t stream) {
  const int rows = 32 / (D / 8);
  const int groups = (a.Hq + rows - 1) / rows + (a.k_new ? 2 * ((a.app.Hkv + rows - 1) / rows) : 0);
  // A warp takes two batches of groups, one group where that leaves the GPU
  // without 16 warps an SM.
  const long long full = static_cast<long long>(num_sms) * 16;
  int parts = (groups + 2 * kRopeBatch - 1) / (2 * kRopeBatch);
  if (static_cast<long long>(a.app.N) * parts < full)
    parts = static_cast<int>(std::min<long long>(groups, (full + a.app.N - 1) / a.app.N));
  a.parts = parts;
  const long long items = static_cast<long long>(a.app.N) * parts;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((items + kRopeThreads / 32 - 1) / (kRopeThreads / 32)));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kv_dtype == PKV_KV_INT8) return launch_rope<128, PKV_KV_INT8>(a, halves, cfg);
  if (kv_dtype == PKV_KV_FP8_E4M3) return launch_rope<128, PKV_KV_FP8_E4M3>(a, halves, cfg);
  return D == 64 ? launch_rope<64, PKV_KV_BF16>(a, halves, cfg) : launch_rope<128, PKV_KV_BF16>(a, halves, cfg);
}

}  // namespace pkv
