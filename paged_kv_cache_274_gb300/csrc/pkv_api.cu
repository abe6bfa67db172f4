// C ABI of the library (see include/pkv.h): host-side validation, tensor-map
// encoding, launch configuration and the sticky device error word.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include <cudaTypedefs.h>

#include "packed_plan.cuh"
#include "pkv_internal.h"
#include "rope_turns.h"

namespace {

// Sticky device error word (PKV_DEVERR_* bits), one per device.
__device__ unsigned int g_pkv_device_error;

thread_local std::string t_last_error;

void set_error(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_last_error = buf;
}

pkv_status fail(pkv_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return st;
}

pkv_status cuda_fail(cudaError_t e, const char* what) {
  return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  void* ctx = nullptr;  // CUDA context the facts below belong to
  unsigned* err_word = nullptr;
  int num_sms = 0;
};
DeviceInfo g_devices[kMaxDevices];
std::mutex g_dev_mutex;

// Per-device facts, resolved with that device current and looked up again
// whenever the device's context changes (a cudaDeviceReset, or a released and
// re-created primary context, loads the module again, possibly at another
// address).
pkv_status device_info(DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(PKV_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  DeviceInfo& d = g_devices[dev];
  void* ctx = pkv::current_context();
  if (ctx == nullptr || ctx != d.ctx) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_pkv_device_error);  // makes the device's context current
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(device error word)");
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
    d.err_word = static_cast<unsigned*>(p);
    d.num_sms = sms;
    d.ctx = pkv::current_context();
  }
  *out = d;
  return PKV_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

pkv_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn) {
  std::call_once(g_encode_once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  if (g_encode == nullptr) return fail(PKV_ERR_CUDA, "driver has no cuTensorMapEncodeTiled");
  *fn = g_encode;
  return PKV_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// page parameters: E4M3 scales are read as floats, INT8 (scale, zero) pairs as float2
bool scales_aligned(int dtype, const void* a, const void* b) {
  const uintptr_t m = dtype == PKV_KV_INT8 ? 7u : 3u;
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & m) == 0;
}

bool aligned4(std::initializer_list<const void*> ps) {
  uintptr_t all = 0;
  for (const void* p : ps) all |= reinterpret_cast<uintptr_t>(p);
  return (all & 3u) == 0;
}

struct Span {
  const void* p;
  size_t bytes;
};

// Rows of `row` bytes, `stride` apart.
struct Rows {
  const void* p;
  int64_t stride, row;
};

// Whether no row of `a` overlaps one of `b` (n of each; NULL: none).  Rows that lie
// between each other's are told apart where both have one stride.
bool rows_disjoint(const Rows& a, const Rows& b, int64_t n) {
  if (a.p == nullptr || b.p == nullptr || n < 1) return true;
  const int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p)), y = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p));
  if (x >= y + (n - 1) * b.stride + b.row || y >= x + (n - 1) * a.stride + a.row) return true;
  if (a.stride != b.stride || n == 1) return false;
  const int64_t off = ((y - x) % a.stride + a.stride) % a.stride;  // of b's rows behind a's
  return off >= a.row && off + b.row <= a.stride;
}

// Whether no array of `written` overlaps another one of them or one of `read`
// (NULL and empty arrays overlap nothing).
bool disjoint(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* v = w + 1; v != written.end(); ++v)
      if (meet(*w, *v)) return false;
    for (const Span& r : read)
      if (meet(*w, r)) return false;
  }
  return true;
}

bool env_flag(const char* name) {
  const char* v = std::getenv(name);
  return v != nullptr && v[0] != '\0' && std::strcmp(v, "0") != 0;
}

int env_int(const char* name, int dflt) {
  const char* v = std::getenv(name);
  if (v == nullptr || v[0] == '\0') return dflt;
  return std::atoi(v);
}

pkv_status check_cache_desc(const pkv_cache_desc* c) {
  if (c == nullptr) return fail(PKV_ERR_INVALID_ARG, "cache descriptor is NULL");
  if (c->num_slots < 1 || c->num_blocks < 1 || c->num_kv_heads < 1)
    return fail(PKV_ERR_INVALID_ARG, "cache: slots, blocks and KV heads must be >= 1");
  if (c->dtype != PKV_KV_BF16 && c->dtype != PKV_KV_FP8_E4M3 && c->dtype != PKV_KV_INT8)
    return fail(PKV_ERR_INVALID_ARG, "cache: unknown dtype %d", c->dtype);
  if (c->block_size != 16 && c->block_size != 32)
    return fail(PKV_ERR_UNSUPPORTED, "cache: block_size %d (supported: 16, 32)", c->block_size);
  if (c->dtype == PKV_KV_BF16 && c->head_dim != 64 && c->head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "cache: head_dim %d (bf16 supports 64, 128)", c->head_dim);
  if (c->dtype != PKV_KV_BF16 && c->head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "cache: head_dim %d (E4M3 and INT8 support 128)", c->head_dim);
  const long long rows = static_cast<long long>(c->num_slots) * c->num_blocks * c->num_kv_heads *
                         c->block_size;
  if (rows >= (1LL << 31)) return fail(PKV_ERR_UNSUPPORTED, "cache has %lld rows (limit 2^31)", rows);
  return PKV_OK;
}

pkv_status encode_cache_map(CUtensorMap* map, const void* base, const pkv_cache_desc* c) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  pkv_status st = tensor_map_encoder(&enc);
  if (st != PKV_OK) return st;
  const bool fp8 = c->dtype != PKV_KV_BF16;  // one-byte elements
  const int elem = fp8 ? 1 : 2;
  const cuuint64_t rows = static_cast<cuuint64_t>(c->num_slots) * c->num_blocks * c->num_kv_heads *
                          c->block_size;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(c->head_dim), rows};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(c->head_dim) * elem};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), static_cast<cuuint32_t>(c->block_size)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return PKV_OK;
}

// Store map of the split-K partial outputs part_o [B][T][Hq][pmax][D] fp32
// for the tcgen05 kernel: a box of 32 columns x one partition x the G heads of
// a KV head x the Tt query tokens of a row tile (128-byte rows, swizzled as
// the kernel stages them); the token dimension clips a ragged last tile.
pkv_status encode_partial_map(CUtensorMap* map, void* part_o, int B, int T, int Hq, int pmax, int D, int G,
                              int Tt) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  pkv_status st = tensor_map_encoder(&enc);
  if (st != PKV_OK) return st;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * sizeof(float);
  cuuint64_t dims[5] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(pmax), static_cast<cuuint64_t>(Hq),
                        static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[4] = {row, row * pmax, row * pmax * Hq, row * pmax * Hq * T};
  cuuint32_t box[5] = {32, 1, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(Tt), 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 5, part_o, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled (partials) failed (%d)", static_cast<int>(r));
  return PKV_OK;
}

// Store map of the bf16 output out [B][T][Hq][D] for the tcgen05 kernel: a
// box of 64 columns x the G heads of a KV head x the Tt query tokens of a row
// tile (128-byte rows, swizzled as the kernel stages them).
pkv_status encode_output_map(CUtensorMap* map, void* out, int B, int T, int Hq, int D, int G, int Tt) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  pkv_status st = tensor_map_encoder(&enc);
  if (st != PKV_OK) return st;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {row, row * Hq, row * Hq * T};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(Tt), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, out, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled (output) failed (%d)", static_cast<int>(r));
  return PKV_OK;
}

// Load map of the queries q [B][T][Hq][D] bf16 for the tile-pair tcgen05
// kernel: a box of 64 columns x the G heads of a KV head x the Tt query
// tokens of a row tile (128-byte rows, 128-byte swizzle, the K-major layout
// of the MMA's A operand); tokens past T read as zeros.
pkv_status encode_query_map(CUtensorMap* map, const void* q, int B, int T, int Hq, int D, int G, int Tt) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  pkv_status st = tensor_map_encoder(&enc);
  if (st != PKV_OK) return st;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {row, row * Hq, row * Hq * T};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(Tt), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled (queries) failed (%d)", static_cast<int>(r));
  return PKV_OK;
}

// Host copies of device tables for PKV_VALIDATE.
template <typename T>
pkv_status fetch(std::vector<T>& dst, const T* src, size_t n, cudaStream_t stream) {
  dst.resize(n);
  if (n == 0) return PKV_OK;
  cudaError_t e = cudaMemcpyAsync(dst.data(), src, n * sizeof(T), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "PKV_VALIDATE copy");
  return PKV_OK;
}

}  // namespace

namespace pkv {
void set_last_error_message(const char* msg) { t_last_error = msg; }

void* current_context() {
  using GetCurrent = CUresult (*)(CUcontext*);
  static GetCurrent fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<GetCurrent>(p);
  }();
  CUcontext ctx = nullptr;
  if (fn == nullptr || fn(&ctx) != CUDA_SUCCESS) return nullptr;
  return ctx;
}
}  // namespace pkv

extern "C" {

int32_t pkv_abi_version(void) { return PKV_ABI_VERSION; }

const char* pkv_status_string(pkv_status s) {
  switch (s) {
    case PKV_OK: return "ok";
    case PKV_ERR_INVALID_ARG: return "invalid argument";
    case PKV_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case PKV_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case PKV_ERR_CUDA: return "CUDA error";
    case PKV_ERR_DEVICE_INDEX: return "device reported an out-of-range index";
    case PKV_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

const char* pkv_last_error_message(void) { return t_last_error.c_str(); }

}  // extern "C"

// What the host can see of a KV append into cache slot `slot` (num_tokens >= 1).
static pkv_status check_append(const pkv_cache_desc* cache, int32_t slot, const void* k, const void* v,
                               const int64_t* slot_mapping, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale) {
  if (slot < 0 || slot >= cache->num_slots)
    return fail(PKV_ERR_INVALID_ARG, "slot %d outside [0, %d)", slot, cache->num_slots);
  const bool fp8 = cache->dtype != PKV_KV_BF16;  // one-byte elements (E4M3 or INT8)
  if (!k || !v || !slot_mapping || !k_cache || !v_cache)
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (fp8 && (!k_scale || !v_scale)) return fail(PKV_ERR_INVALID_ARG, "E4M3 and INT8 caches need k_scale and v_scale");
  if (fp8 && !scales_aligned(cache->dtype, k_scale, v_scale))
    return fail(PKV_ERR_ALIGNMENT, "k_scale and v_scale must be 4-byte (E4M3) or 8-byte (INT8) aligned");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(PKV_ERR_ALIGNMENT, "k, v and caches must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
    return fail(PKV_ERR_ALIGNMENT, "slot_mapping must be 8-byte aligned");
  return PKV_OK;
}

// Validate a KV append into cache slot `slot` and resolve its launch
// arguments; *a is left untouched unless PKV_OK.  num_tokens >= 1.
static pkv_status prepare_append(const pkv_cache_desc* cache, int32_t slot, const void* k, const void* v,
                                 const int64_t* slot_mapping, int32_t num_tokens, void* k_cache,
                                 void* v_cache, const float* k_scale, const float* v_scale,
                                 cudaStream_t s, const DeviceInfo* dev, pkv::AppendArgs* a) {
  pkv_status st = check_append(cache, slot, k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale);
  if (st != PKV_OK) return st;
  const bool fp8 = cache->dtype != PKV_KV_BF16;  // one-byte elements (E4M3 or INT8)
  const long long nslots = static_cast<long long>(cache->num_blocks) * cache->block_size;
  if (env_flag("PKV_VALIDATE")) {
    std::vector<int64_t> sm;
    if ((st = fetch(sm, slot_mapping, static_cast<size_t>(num_tokens), s)) != PKV_OK) return st;
    std::vector<int64_t> seen;
    for (int i = 0; i < num_tokens; ++i) {
      if (sm[i] < -1 || sm[i] >= nslots)
        return fail(PKV_ERR_INVALID_ARG, "slot_mapping[%d] = %lld outside [-1, %lld)", i,
                    static_cast<long long>(sm[i]), nslots);
      if (sm[i] >= 0) seen.push_back(sm[i]);
    }
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end())
      return fail(PKV_ERR_INVALID_ARG, "slot_mapping has duplicate slots");
  }
  const size_t page_elems = static_cast<size_t>(cache->num_kv_heads) * cache->block_size * cache->head_dim;
  const size_t slot_elems = page_elems * cache->num_blocks;
  const size_t elem = fp8 ? 1 : 2;
  const size_t scale_off = static_cast<size_t>(slot) * cache->num_blocks * cache->num_kv_heads *
                           (cache->dtype == PKV_KV_INT8 ? 2 : 1);
  a->k = static_cast<const uint4*>(k);
  a->v = static_cast<const uint4*>(v);
  a->slot_mapping = slot_mapping;
  a->N = num_tokens;
  a->Hkv = cache->num_kv_heads;
  a->D = cache->head_dim;
  a->bs = cache->block_size;
  a->nslots = nslots;
  a->kc = static_cast<uint8_t*>(k_cache) + static_cast<size_t>(slot) * slot_elems * elem;
  a->vc = static_cast<uint8_t*>(v_cache) + static_cast<size_t>(slot) * slot_elems * elem;
  a->ks = fp8 ? k_scale + scale_off : nullptr;
  a->vs = fp8 ? v_scale + scale_off : nullptr;
  a->err = dev->err_word;
  return PKV_OK;
}

extern "C" {

pkv_status pkv_kv_append(const pkv_cache_desc* cache, int32_t slot, const void* k, const void* v,
                         const int64_t* slot_mapping, int32_t num_tokens, void* k_cache,
                         void* v_cache, const float* k_scale, const float* v_scale, void* stream) {
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (slot < 0 || slot >= cache->num_slots)
    return fail(PKV_ERR_INVALID_ARG, "slot %d outside [0, %d)", slot, cache->num_slots);
  if (num_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens %d < 0", num_tokens);
  if (num_tokens == 0) return PKV_OK;
  if ((st = check_append(cache, slot, k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale)) != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev_info;
  const DeviceInfo* dev = &dev_info;
  if ((st = device_info(&dev_info)) != PKV_OK) return st;
  pkv::AppendArgs a{};
  if ((st = prepare_append(cache, slot, k, v, slot_mapping, num_tokens, k_cache, v_cache, k_scale, v_scale, s,
                           dev, &a)) != PKV_OK)
    return st;
  cudaError_t e = pkv::launch_kv_append(cache->dtype, a, s);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
  return PKV_OK;
}

pkv_status pkv_rope_append(const pkv_cache_desc* cache, int32_t slot, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const void* v, int64_t v_stride, int32_t num_tokens, int32_t num_q_heads,
                           const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                           int32_t num_axes, const double* inv_freq, const int32_t* freq_axes, int32_t rotary_dim,
                           int32_t interleaved, const int64_t* slot_mapping, void* q_out, int64_t q_out_stride,
                           void* k_cache, void* v_cache, const float* k_scale, const float* v_scale, void* stream) {
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  const int D = cache->head_dim, R = rotary_dim, N = num_tokens;
  if (slot < 0 || slot >= cache->num_slots)
    return fail(PKV_ERR_INVALID_ARG, "slot %d outside [0, %d)", slot, cache->num_slots);
  if (N < 0) return fail(PKV_ERR_INVALID_ARG, "num_tokens %d < 0", N);
  if (num_q_heads < 1) return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d < 1", num_q_heads);
  if (R < 0 || R > D || R % 16 != 0)
    return fail(PKV_ERR_UNSUPPORTED, "rotary_dim %d (supported: multiples of 16 up to the head_dim %d)", R, D);
  if (interleaved != 0 && interleaved != 1) return fail(PKV_ERR_INVALID_ARG, "interleaved %d", interleaved);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(PKV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((k == nullptr) != (v == nullptr)) return fail(PKV_ERR_INVALID_ARG, "k and v go together");
  const bool append = k != nullptr;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * D, kv_row = static_cast<int64_t>(cache->num_kv_heads) * D;
  if (q_row >= (1LL << 31)) return fail(PKV_ERR_UNSUPPORTED, "num_q_heads %d", num_q_heads);
  // (then the kernel's items, at most half a part for 8 heads, fit 31 bits)
  if (N * (num_q_heads + 2LL * cache->num_kv_heads) >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "%d tokens of %d and %d heads", N, num_q_heads, cache->num_kv_heads);
  if (q_stride < q_row || q_out_stride < q_row || (append && (k_stride < kv_row || v_stride < kv_row)))
    return fail(PKV_ERR_INVALID_ARG, "a token stride is below the size of its heads");
  if ((q_stride | q_out_stride) % 8 != 0 || (append && (k_stride | v_stride) % 8 != 0))
    return fail(PKV_ERR_ALIGNMENT, "token strides must be multiples of 8 elements");
  const int64_t strides = std::max(std::max(q_stride, q_out_stride), append ? std::max(k_stride, v_stride) : 0);
  if (strides >= (1LL << 31)) return fail(PKV_ERR_UNSUPPORTED, "token stride %lld", static_cast<long long>(strides));
  if (R > 0) {
    if (num_axes < 1 || num_axes > PKV_MAX_POSITION_AXES)
      return fail(PKV_ERR_INVALID_ARG, "num_axes %d outside 1..%d", num_axes, PKV_MAX_POSITION_AXES);
    if (inv_freq == nullptr) return fail(PKV_ERR_INVALID_ARG, "inv_freq is NULL");
    for (int i = 0; i < R / 2; ++i) {
      if (!std::isfinite(inv_freq[i])) return fail(PKV_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
      if (freq_axes != nullptr && (freq_axes[i] < 0 || freq_axes[i] >= num_axes))
        return fail(PKV_ERR_INVALID_ARG, "freq_axes[%d] = %d outside [0, %d)", i, freq_axes[i], num_axes);
    }
  }
  if (N == 0) return PKV_OK;
  if (!q || !q_out || (R > 0 && !positions) || (append && !slot_mapping))
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(q_weight) || !aligned16(k_weight))
    return fail(PKV_ERR_ALIGNMENT, "q, q_out and the norms' weights must be 16-byte aligned");
  if (!aligned4({positions}) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
    return fail(PKV_ERR_ALIGNMENT, "positions must be 4-byte aligned, slot_mapping 8-byte");
  if (append && (st = check_append(cache, slot, k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale)) != PKV_OK) return st;
  const Rows out_rows{q_out, 2 * q_out_stride, 2 * q_row}, q_rows{q, 2 * q_stride, 2 * q_row};
  const Rows k_rows{k, 2 * k_stride, 2 * kv_row}, v_rows{v, 2 * v_stride, 2 * kv_row};
  const bool in_place = q_out == q && q_out_stride == q_stride;
  const size_t pool = static_cast<size_t>(cache->num_slots) * cache->num_blocks * cache->num_kv_heads * cache->block_size * D *
                      (cache->dtype == PKV_KV_BF16 ? 2 : 1);
  const size_t weights = static_cast<size_t>(D) * 2, rows = static_cast<size_t>(N);
  const Span none{nullptr, 0};
  // (q_out may lie between the rows of q, k and v: in place it does where they are one projection's)
  if ((!in_place && !rows_disjoint(out_rows, q_rows, N)) || !rows_disjoint(out_rows, k_rows, N) || !rows_disjoint(out_rows, v_rows, N) ||
      !disjoint({Span{q_out, static_cast<size_t>((N - 1) * 2 * q_out_stride + 2 * q_row)}},
                {Span{q_weight, weights}, Span{k_weight, weights},
                 R > 0 ? Span{positions, rows * 4 * num_axes} : none, Span{slot_mapping, rows * 8},
                 append ? Span{k_cache, pool} : none, append ? Span{v_cache, pool} : none}))
    return fail(PKV_ERR_INVALID_ARG, "q_out overlaps another array");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if ((st = device_info(&dev)) != PKV_OK) return st;
  pkv::RopeArgs a{};
  if (append) {
    if ((st = prepare_append(cache, slot, k, v, slot_mapping, N, k_cache, v_cache, k_scale, v_scale, s, &dev, &a.app)) != PKV_OK)
      return st;
  } else {
    a.app.N = N;
    a.app.Hkv = cache->num_kv_heads;
    a.app.D = D;
    a.app.bs = cache->block_size;
    a.app.nslots = static_cast<int64_t>(cache->num_blocks) * cache->block_size;
    a.app.slot_mapping = slot_mapping;
    a.app.err = dev.err_word;
  }
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.qw = static_cast<const uint16_t*>(q_weight);
  a.kw = append ? static_cast<const uint16_t*>(k_weight) : nullptr;
  a.positions = positions;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.out_stride = q_out_stride;
  a.eps = eps;
  a.Hq = num_q_heads;
  a.R = R;
  a.k_new = append ? 1 : 0;
  for (int i = 0; i < R / 2; ++i) {
    a.turns[i] = pkv::rope_turns(inv_freq[i]);
    a.axis[i] = static_cast<uint8_t>(freq_axes != nullptr ? freq_axes[i] : 0);
  }
  cudaError_t e = pkv::launch_rope_append(cache->dtype, D, interleaved == 0, a, dev.num_sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "rope_append launch");
  return PKV_OK;
}

// Resolve options into a full launch configuration (no device work).
static pkv_status resolve_decode(const pkv_cache_desc* c, int32_t batch, int32_t T, int32_t Hq,
                                 int32_t MB, const pkv_decode_opts* opts, int num_sms,
                                 pkv::DecodeLaunch* L, bool tree = false) {
  pkv_status st = check_cache_desc(c);
  if (st != PKV_OK) return st;
  if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (T < 1 || T > PKV_MAX_QUERY_TOKENS)
    return fail(PKV_ERR_INVALID_ARG, "num_query_tokens %d outside 1..%d", T, PKV_MAX_QUERY_TOKENS);
  if (MB < 1) return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d < 1", MB);
  if (Hq < 1 || Hq % c->num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d", Hq,
                c->num_kv_heads);
  if (static_cast<long long>(MB) * c->block_size >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  const int G = Hq / c->num_kv_heads;
  pkv_decode_opts o{};
  if (opts) o = *opts;
  int math = o.math != 0 ? o.math : env_int("PKV_DECODE_MATH", PKV_MATH_AUTO);
  // tcgen05 tiles: multi-token calls with head_dim 128 (one-byte caches as
  // exact code values: E4M3 K pages as they are, the other pages widened to
  // f16 in shared memory)
  // (drafted trees: head_dim 64 and single nodes too)
  const bool tc_ok = tree ? G <= 128 : c->head_dim == 128 && T > 1 && G <= 128;
  // measured on GB300 (Llama-8B layer, G 4): mma.sync tiles are faster up to
  // 16 rows per KV head (172 us at 4 tokens, one tile), tcgen05 tiles from 32
  // rows on (kernel 173 vs 234 us at 8 tokens, 173 vs 451 at 16, 183 vs 865
  // at 32, 583 vs 3402 at 128)
  // drafted trees, 8 KV heads, mma.sync against tcgen05, us a call: bf16 with
  // head_dim 128 no case for mma.sync from 8 rows on (64 x 4096 tokens 174 vs 173,
  // 16 x 1024 34 vs 26, 1 x 16384 26 vs 27); head_dim 64 up to 8 rows (64 x 4096:
  // 91 vs 105, 12 rows: 104 vs 104, and 28 vs 21 for 16 x 1024); one-byte caches up
  // to 16 rows, which is right for large batches (64 x 4096: E4M3 156 vs 160, INT8
  // 148 vs 202; 20 rows: 266 vs 160, 252 vs 202) and for long single requests (1 x
  // 16384: 29 vs 29, 29 vs 32), while 16 x 1024 would be faster with tcgen05 from 8
  // rows on (E4M3 33 vs 29; INT8 31 vs 32, 12 rows: 36 vs 32)
  const long long mma_rows = !tree || c->dtype != PKV_KV_BF16 ? 16 : c->head_dim == 64 ? 8 : 0;
  if (math == PKV_MATH_AUTO) math = (tc_ok && static_cast<long long>(T) * G > mma_rows) ? PKV_MATH_TC : PKV_MATH_MMA;
  if (math == PKV_MATH_TC && !tc_ok)
    return tree ? fail(PKV_ERR_UNSUPPORTED, "G = %d query heads per KV head (tcgen05 tiles of drafted trees support <= 128)", G)
                : fail(PKV_ERR_UNSUPPORTED, "tcgen05 tiles need T > 1, head_dim 128 and G <= 128");
  if (math == PKV_MATH_MMA && G > 16)
    return fail(PKV_ERR_UNSUPPORTED, "G = %d query heads per KV head (mma supports <= 16)", G);
  if (math == PKV_MATH_FFMA && G != 1 && G != 2 && G != 4 && G != 8)
    return fail(PKV_ERR_UNSUPPORTED, "G = %d query heads per KV head (ffma supports 1, 2, 4, 8)", G);
  if (math != PKV_MATH_MMA && math != PKV_MATH_FFMA && math != PKV_MATH_TC)
    return fail(PKV_ERR_INVALID_ARG, "math %d", math);
  const bool tc = math == PKV_MATH_TC;
  if (math == PKV_MATH_FFMA && (T > 1 || tree))
    return fail(PKV_ERR_UNSUPPORTED, tree ? "drafted trees need the mma.sync or the tcgen05 back-end"
                                          : "multi-token queries need the mma back-end");
  if (static_cast<long long>(batch) * T * Hq * c->head_dim >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "batch x query tokens x heads x head_dim too large");
  // row tiles of at most 16 (mma.sync) or 128 (tcgen05) (query token, head)
  // rows: whole query tokens per tile
  const int Tt = std::max(1, std::min(T, (tc ? 128 : 16) / G));
  const int NT = (T + Tt - 1) / Tt;
  const bool fp8 = c->dtype != PKV_KV_BF16;  // one-byte elements
  const size_t stage_bytes = static_cast<size_t>(2) * c->block_size * c->head_dim * (fp8 ? 1 : 2);
  // Defaults measured on GB300: 4 warps per CTA with shallow (2-stage)
  // rings give several CTAs, i.e. 8+ streaming warps, per SM; deeper rings
  // only cost occupancy.
  // (the tcgen05 kernels have fixed shapes: one 128-row tile per CTA with 4
  // compute warps, an MMA warp and two copy warps, a 4-stage K ring and a
  // 2-stage V ring of 64 tokens; or, with two or more row tiles per KV head,
  // a pair of tiles per CTA with 8 softmax warps, an MMA warp and two copy
  // warps, 2-stage K and V rings of 128 tokens -- PKV_TC_PAIR=0 keeps the
  // one-tile kernel there)
  const bool tc2 = tc && !tree && NT >= 2 && c->dtype == PKV_KV_BF16 && env_int("PKV_TC_PAIR", 1) != 0;
  // drafted trees on tcgen05 (tree_attend.cuh): one CTA per SM, one or a pair
  // of row tiles each, equal shares of 128-token steps instead of partitions
  const bool tree_tc = tree && tc;
  int warps = tc2 ? pkv::kTcPairWarps
              : tc ? (c->dtype == PKV_KV_BF16 ? 7 : 8)  // + the converter warp of one-byte caches
                   : (o.warps_per_cta != 0 ? o.warps_per_cta : env_int("PKV_DECODE_WARPS", 4));
  int stages = tc2 ? 2 : tc ? 4 : (o.stages != 0 ? o.stages : env_int("PKV_DECODE_STAGES", 0));
  if (stages == 0) stages = stage_bytes >= (8u << 10) ? 2 : 3;
  if (!tc && (warps < 1 || warps > 8)) return fail(PKV_ERR_INVALID_ARG, "warps_per_cta %d outside 1..8", warps);
  if (stages < 2 || stages > 8) return fail(PKV_ERR_INVALID_ARG, "stages %d outside 2..8", stages);
  if (tree_tc) {
    warps = c->dtype == PKV_KV_BF16 ? 20 : 28;
    stages = 2;
  }
  const size_t smem = tree_tc ? pkv::tree_attend_smem_bytes(c->dtype, c->head_dim, NT > 1)
                              : pkv::decode_smem_bytes(fp8, c->head_dim, c->block_size, warps, stages, tc, tc2);
  if (smem > 227u * 1024u)
    return fail(PKV_ERR_INVALID_ARG, "warps x stages need %zu bytes of shared memory", smem);
  int ppu = o.partition_blocks != 0 ? o.partition_blocks : env_int("PKV_DECODE_PARTITION_BLOCKS", 0);
  // partitions of up to 64 blocks for the mma.sync kernels, up to a unit's
  // page table for the tcgen05 kernel
  const int ppu_max = tc ? pkv::kTcUnitMaxPages : 64;
  if (ppu < 0 || ppu > ppu_max) return fail(PKV_ERR_INVALID_ARG, "partition_blocks %d outside 1..%d", ppu, ppu_max);
  const bool auto_ppu = ppu == 0;
  const int tree_min_blocks = ppu;
  if (tree_tc) {
    ppu = MB;  // no partitions of a fixed length
  } else if (ppu == 0) {
    // The decode is a persistent grid of W streaming warps pulling units of
    // work; its time follows how full the last round of units is.  Estimate
    // W from shared memory and about 200 registers a thread, count units for
    // the longest allowed context, take 64-block partitions when one round
    // holds every unit, else the size of {32, 16, 8} whose last round is
    // fullest (a larger size unless a smaller one is clearly better).
    const long long ctas_smem = std::max<long long>(1, (228LL * 1024) / static_cast<long long>(smem + 1024));
    const long long ctas_regs = std::max<long long>(1, 65536LL / (warps * 32LL * 200));
    // streams: warps of the mma.sync kernels; CTAs of the tcgen05 kernel
    // (two per SM: their accumulators fill the SM's tensor memory)
    const long long W = tc2 ? static_cast<long long>(num_sms)
                        : tc ? 2LL * num_sms
                             : static_cast<long long>(num_sms) * std::min(ctas_smem, ctas_regs) * warps;
    const int tiles_per_unit = tc2 ? 2 : 1;
    auto units = [&](int pp) {
      return static_cast<long long>(std::max(batch, 1)) * c->num_kv_heads * ((NT + tiles_per_unit - 1) / tiles_per_unit) *
             ((MB + pp - 1) / pp);
    };
    // Multi-token units carry T times the partials and load up to 16 query
    // rows each, so they stay at 32 or 64 blocks (measured on the 4- and
    // 8-token verify steps: 32 beats 16 by 4-10% in the kernel).
    const std::vector<int> sizes = T > 1 ? std::vector<int>{32, 64} : std::vector<int>{32, 16, 8};
    if (tc) {
      // tcgen05 units cost their 64-token steps plus a start-up and write-out
      // of about 6.5 steps (measured on GB300); rounds of 2 x SMs units:
      // the size of {64, 128, 256} blocks with the least modelled time
      // (long units also drop the split-K partials and the merge)
      // A sequence in several partitions also writes split-K partials that
      // the merge kernel reads back: (query rows) x (D + 2) fp32 per unit,
      // each way, at about 4 MB per modelled step (measured on GB300: the
      // 64-token verify step with 128-block units ran 393 us against 345
      // with whole-sequence units, whose kernel alone is 18 us slower).
      // The tile-pair kernel: steps of 128 tokens for two tiles, i.e. about
      // two 64-token steps of the one-tile kernel, and units twice as wide.
      const double partial_bytes = static_cast<double>(G) * Tt * (c->head_dim + 2) * 4.0 * tiles_per_unit;
      double best = 0.0;
      for (int pp : {64, 128, 256}) {
        const long long rounds = (units(pp) + W - 1) / W;
        const double merge = pp < MB ? static_cast<double>(units(pp)) * partial_bytes * 2.0 / 4.0e6 : 0.0;
        const double cost = static_cast<double>(rounds) *
                            (static_cast<double>(pp) * c->block_size / 64.0 + 6.5) + merge;
        if (best == 0.0 || cost < best) {
          best = cost;
          ppu = pp;
        }
        if (pp >= MB) break;  // one partition per sequence already
      }
    } else if (units(64) <= W) {
      // one round holds every unit: cut the sequences so that each SM gets
      // the same number of units, one per warp of a CTA per SM (measured on
      // GB300: 64-block units of the 70B-shaped 32K x 4 and 128K x 1 contexts
      // filled 128 CTAs of 4 warps on 152 SMs), in partitions of 16 to 64
      // blocks
      const long long seq_units = static_cast<long long>(std::max(batch, 1)) * c->num_kv_heads * NT;
      const long long parts = std::max<long long>((MB + 63) / 64, (static_cast<long long>(num_sms) * warps) / seq_units);
      ppu = static_cast<int>(std::min<long long>(64, std::max<long long>(16, (MB + parts - 1) / parts)));
    } else {
      double best = -1.0;
      for (int pp : sizes) {
        const double r = static_cast<double>(units(pp)) / static_cast<double>(W);
        const double eff = r / std::ceil(r);
        if (eff > best + 0.05) {
          best = eff;
          ppu = pp;
        }
      }
    }
  }
  ppu = std::min(ppu, MB);
  if (!tree_tc && (MB + ppu - 1) / ppu > 65536)
    return fail(PKV_ERR_UNSUPPORTED, "more than 65536 partitions per sequence; raise partition_blocks");
  // The tile-pair kernel runs one unit per SM at a time, units of equal
  // length: when the last round of units would be at most half full, the
  // last sequences take partitions of half the length, so that the last
  // round's work spreads over twice as many units (with S sequences halved,
  // S >= r / u: the r units of the last round become at least 2r half
  // units).  Counted for sequences of the longest allowed context; with
  // shorter ones the split is still valid, only less useful.
  int half_from = batch, ppu_half = ppu;
  if (tc2 && auto_ppu && ppu >= 2 && env_int("PKV_TC_BALANCE", 1) != 0) {
    const long long u = static_cast<long long>((MB + ppu - 1) / ppu) * c->num_kv_heads * ((NT + 1) / 2);
    const long long n = static_cast<long long>(std::max(batch, 1)) * u;
    const long long r = n % num_sms;
    if (r > 0 && 2 * r <= num_sms) {
      half_from = batch - static_cast<int>(std::min<long long>(batch, (r + u - 1) / u));
      ppu_half = (ppu + 1) / 2;
    }
  }
  *L = pkv::DecodeLaunch{};
  L->tree = tree ? 1 : 0;
  L->tree_words = tree ? (T + 31) / 32 : 0;
  if (tree_tc) {
    L->tree_tc = 1;
    // pairs of row tiles side by side: the CTAs of one share read the same
    // pages, at the same time
    L->tree_shares = std::max(1, num_sms / (NT > 1 ? (NT + 1) / 2 : 1));
    L->tree_min_steps = std::max(1, tree_min_blocks * c->block_size / 128);
  }
  if (tree && static_cast<long long>(batch) * L->tree_words * std::max(T, c->num_kv_heads) >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "batch x nodes x mask words too large");
  L->B = batch;
  L->Hq = Hq;
  L->Hkv = c->num_kv_heads;
  L->G = G;
  L->T = T;
  L->Tt = Tt;
  L->NT = NT;
  L->tc = tc ? 1 : 0;
  L->tc2 = tc2 ? 1 : 0;
  L->MB = MB;
  L->NB = c->num_blocks;
  L->bs = c->block_size;
  L->D = c->head_dim;
  L->kv_fp8 = fp8;
  L->kv_dtype = c->dtype;
  L->ppu = ppu;
  L->half_from = half_from;
  L->ppu_half = ppu_half;
  L->pmax = (MB + ppu_half - 1) / ppu_half;  // ppu_half == ppu without half-length partitions
  L->math = math;
  L->warps = warps;
  L->stages = stages;
  L->num_sms = num_sms;
  return PKV_OK;
}

// Likewise for packed rows: N rows of `batch` sequences, at most T of each.
static pkv_status resolve_packed(const pkv_cache_desc* c, int32_t N, int32_t batch, int32_t T, int32_t Hq, int32_t MB,
                                 const pkv_decode_opts* opts, pkv::DecodeLaunch* L) {
  pkv_status st = check_cache_desc(c);
  if (st != PKV_OK) return st;
  if (batch < 0 || N < 0) return fail(PKV_ERR_INVALID_ARG, "batch %d, num_rows %d < 0", batch, N);
  if (T < 1) return fail(PKV_ERR_INVALID_ARG, "max_query_tokens %d < 1", T);
  if (MB < 1) return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d < 1", MB);
  if (Hq < 1 || Hq % c->num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARG, "num_q_heads %d is not a multiple of num_kv_heads %d", Hq, c->num_kv_heads);
  if (static_cast<long long>(MB) * c->block_size >= (1LL << 31) - 256 || static_cast<long long>(batch) * MB >= (1LL << 40))
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  const int G = Hq / c->num_kv_heads;
  if (G > 128) return fail(PKV_ERR_UNSUPPORTED, "G = %d query heads per KV head (packed rows support <= 128)", G);
  pkv_decode_opts o{};
  if (opts) o = *opts;
  if (o.math != PKV_MATH_AUTO && o.math != PKV_MATH_TC)
    return fail(PKV_ERR_UNSUPPORTED, "math %d (packed rows have the tcgen05 back-end only)", o.math);
  if (o.partition_blocks < 0 || o.partition_blocks > pkv::kTcUnitMaxPages)
    return fail(PKV_ERR_INVALID_ARG, "partition_blocks %d outside 1..%d", o.partition_blocks, pkv::kTcUnitMaxPages);
  if (static_cast<long long>(N) * Hq * c->head_dim >= (1LL << 31) || static_cast<long long>(N) * c->num_kv_heads >= (1LL << 31) || batch >= (1 << 24))
    return fail(PKV_ERR_UNSUPPORTED, "rows x heads x head_dim or batch too large");
  *L = pkv::DecodeLaunch{};
  L->packed = 1;
  L->N = N;
  L->B = batch;
  L->Hq = Hq;
  L->Hkv = c->num_kv_heads;
  L->G = G;
  L->T = std::min(T, std::max(N, 1));
  // tiles of 128 (row, head) rows; a pair of them per CTA where a sequence may
  // have more than one
  L->Tt = std::max(1, std::min(L->T, 128 / G));
  L->NT = L->T > L->Tt ? 2 : 1;
  L->MB = MB;
  L->NB = c->num_blocks;
  L->bs = c->block_size;
  L->D = c->head_dim;
  L->kv_fp8 = c->dtype != PKV_KV_BF16;
  L->kv_dtype = c->dtype;
  L->math = PKV_MATH_TC;
  L->tree_shares = pkv::kPackedShares;
  L->tree_min_steps = std::max(1, o.partition_blocks * c->block_size / 128);
  return PKV_OK;
}

static size_t packed_total(const pkv::DecodeLaunch& L) {
  return pkv::packed_workspace(L.B, L.N, L.Hkv, L.D, L.NT, L.tree_shares).total;
}

static size_t workspace_total(const pkv::DecodeLaunch& L) {
  if (L.tree_tc) return pkv::tree_workspace(L.B, L.Hkv, L.D, L.NT, L.tree_words, L.tree_shares).total;
  return pkv::workspace_layout(L.B, L.T, L.Hq, L.Hkv, L.NT, L.D, L.pmax, L.tree_words).total;
}

static pkv::WorkspaceLayout layout_of(const pkv::DecodeLaunch& L) {
  return pkv::workspace_layout(L.B, L.T, L.Hq, L.Hkv, L.NT, L.D, L.pmax, L.tree_words);
}

static size_t workspace_bytes_of(const pkv_cache_desc* cache, int32_t batch, int32_t num_query_tokens,
                                 int32_t num_q_heads, int32_t max_blocks_per_seq,
                                 const pkv_decode_opts* opts, bool tree) {
  pkv::DecodeLaunch L;
  // The partition size (and so the workspace) must not depend on the device
  // the call later runs on: size with the largest SM count this build targets.
  if (resolve_decode(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts, 152, &L, tree) !=
      PKV_OK)
    return 0;
  return workspace_total(L);
}

size_t pkv_decode_multi_workspace_bytes(const pkv_cache_desc* cache, int32_t batch,
                                        int32_t num_query_tokens, int32_t num_q_heads,
                                        int32_t max_blocks_per_seq, const pkv_decode_opts* opts) {
  return workspace_bytes_of(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts, false);
}

size_t pkv_decode_tree_workspace_bytes(const pkv_cache_desc* cache, int32_t batch,
                                       int32_t num_query_tokens, int32_t num_q_heads,
                                       int32_t max_blocks_per_seq, const pkv_decode_opts* opts) {
  return workspace_bytes_of(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts, true);
}

size_t pkv_decode_packed_workspace_bytes(const pkv_cache_desc* cache, int32_t num_rows, int32_t batch,
                                         int32_t max_query_tokens, int32_t num_q_heads,
                                         int32_t max_blocks_per_seq, const pkv_decode_opts* opts) {
  pkv::DecodeLaunch L;
  if (resolve_packed(cache, num_rows, batch, max_query_tokens, num_q_heads, max_blocks_per_seq, opts, &L) != PKV_OK) return 0;
  return packed_total(L);
}

size_t pkv_decode_workspace_bytes(const pkv_cache_desc* cache, int32_t batch, int32_t num_q_heads,
                                  int32_t max_blocks_per_seq, const pkv_decode_opts* opts) {
  return pkv_decode_multi_workspace_bytes(cache, batch, 1, num_q_heads, max_blocks_per_seq, opts);
}

static pkv_status describe(const pkv_cache_desc* cache, int32_t batch, int32_t num_query_tokens,
                           int32_t num_q_heads, int32_t max_blocks_per_seq, const pkv_decode_opts* opts,
                           pkv_decode_plan* plan, bool tree) {
  if (plan == nullptr) return fail(PKV_ERR_INVALID_ARG, "plan is NULL");
  pkv::DecodeLaunch L;
  pkv_status st = resolve_decode(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts,
                                 152, &L, tree);
  if (st != PKV_OK) return st;
  plan->partition_blocks = L.ppu;
  plan->max_partitions = L.pmax;
  plan->math = L.math;
  plan->warps_per_cta = L.warps;
  plan->stages = L.stages;
  // the merge kernel runs above 4 partitions (tcgen05 kernel: above 1)
  plan->kernels_per_call = L.pmax > (L.tc ? 1 : 4) ? 3 : 2;
  if (L.tree_tc) plan->kernels_per_call = L.tree_shares > 1 ? 3 : 2;
  plan->workspace_bytes = workspace_total(L);
  plan->smem_bytes_per_cta = L.tree_tc ? pkv::tree_attend_smem_bytes(L.kv_dtype, L.D, L.NT > 1)
                                       : pkv::decode_smem_bytes(L.kv_fp8, L.D, L.bs, L.warps, L.stages, L.tc, L.tc2);
  plan->query_tokens_per_tile = L.Tt;
  plan->row_tiles = L.NT;
  return PKV_OK;
}

pkv_status pkv_decode_multi_describe(const pkv_cache_desc* cache, int32_t batch,
                                     int32_t num_query_tokens, int32_t num_q_heads,
                                     int32_t max_blocks_per_seq, const pkv_decode_opts* opts,
                                     pkv_decode_plan* plan) {
  return describe(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts, plan, false);
}

pkv_status pkv_decode_tree_describe(const pkv_cache_desc* cache, int32_t batch,
                                    int32_t num_query_tokens, int32_t num_q_heads,
                                    int32_t max_blocks_per_seq, const pkv_decode_opts* opts,
                                    pkv_decode_plan* plan) {
  return describe(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts, plan, true);
}

pkv_status pkv_decode_describe(const pkv_cache_desc* cache, int32_t batch, int32_t num_q_heads,
                               int32_t max_blocks_per_seq, const pkv_decode_opts* opts,
                               pkv_decode_plan* plan) {
  return pkv_decode_multi_describe(cache, batch, 1, num_q_heads, max_blocks_per_seq, opts, plan);
}

}  // extern "C"

// The new tokens of a fused append-and-decode call.
struct AppendRequest {
  const void* k;
  const void* v;
  const int64_t* slot_mapping;
  int32_t num_tokens;
};

// The trees of a drafted-tree call.
struct TreeRequest {
  const uint32_t* mask;
  int32_t tree_batch;
  const int32_t* node_counts;
};

static pkv_status decode_call(const pkv_cache_desc* cache, const void* q, int32_t batch,
                              int32_t num_query_tokens, int32_t num_q_heads, const void* k_cache,
                              const void* v_cache, const float* k_scale, const float* v_scale,
                              const int32_t* block_tables, int32_t max_blocks_per_seq,
                              const int32_t* context_lens, const int32_t* kv_group_ptr,
                              int32_t num_layers, int32_t layer, float scale, void* out,
                              void* workspace, size_t workspace_bytes,
                              const pkv_decode_opts* opts, void* stream, const AppendRequest* req,
                              const TreeRequest* tree = nullptr) {
  pkv::DecodeLaunch L;
  pkv_status st = resolve_decode(cache, batch, num_query_tokens, num_q_heads, max_blocks_per_seq, opts,
                                 152, &L, tree != nullptr);
  if (st != PKV_OK) return st;
  if (tree != nullptr && tree->tree_batch != 1 && tree->tree_batch != batch)
    return fail(PKV_ERR_INVALID_ARG, "tree_batch %d is neither 1 nor the batch %d", tree->tree_batch, batch);
  if (kv_group_ptr == nullptr || num_layers < 1 || layer < 0 || layer >= num_layers)
    return fail(PKV_ERR_INVALID_ARG, "layer %d / num_layers %d / kv_group_ptr", layer, num_layers);
  const int32_t slot = kv_group_ptr[layer];
  if (slot < 0 || slot >= cache->num_slots)
    return fail(PKV_ERR_INVALID_ARG, "kv_group_ptr[%d] = %d outside [0, %d)", layer, slot, cache->num_slots);
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (batch == 0) {  // nothing to decode: only the append, if any
    if (req == nullptr || req->num_tokens == 0) return PKV_OK;
    return pkv_kv_append(cache, slot, req->k, req->v, req->slot_mapping, req->num_tokens,
                         const_cast<void*>(k_cache), const_cast<void*>(v_cache), k_scale, v_scale, stream);
  }
  const bool fp8 = cache->dtype != PKV_KV_BF16;  // one-byte elements (E4M3 or INT8)
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (fp8 && (!k_scale || !v_scale)) return fail(PKV_ERR_INVALID_ARG, "E4M3 and INT8 caches need k_scale and v_scale");
  if (fp8 && !scales_aligned(cache->dtype, k_scale, v_scale))
    return fail(PKV_ERR_ALIGNMENT, "k_scale and v_scale must be 4-byte (E4M3) or 8-byte (INT8) aligned");
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace))
    return fail(PKV_ERR_ALIGNMENT, "q, out, caches and workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return fail(PKV_ERR_ALIGNMENT, "block_tables and context_lens must be 4-byte aligned");
  if (tree != nullptr) {
    if (tree->mask == nullptr) return fail(PKV_ERR_INVALID_ARG, "tree_mask is NULL");
    if ((reinterpret_cast<uintptr_t>(tree->mask) & 3u) || (reinterpret_cast<uintptr_t>(tree->node_counts) & 3u))
      return fail(PKV_ERR_ALIGNMENT, "tree_mask and node_counts must be 4-byte aligned");
  }
  const size_t qbytes = static_cast<size_t>(batch) * num_query_tokens * num_q_heads * cache->head_dim * 2;
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  if (qa < oa + qbytes && oa < qa + qbytes) return fail(PKV_ERR_INVALID_ARG, "out overlaps q");
  const size_t need = workspace_total(L);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
  const pkv::WorkspaceLayout wl = layout_of(L);

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev_info;
  const DeviceInfo* dev = &dev_info;
  if ((st = device_info(&dev_info)) != PKV_OK) return st;
  L.num_sms = dev->num_sms;

  if (env_flag("PKV_VALIDATE")) {
    std::vector<int32_t> ctx, bt;
    if ((st = fetch(ctx, context_lens, static_cast<size_t>(batch), s)) != PKV_OK) return st;
    if ((st = fetch(bt, block_tables, static_cast<size_t>(batch) * max_blocks_per_seq, s)) != PKV_OK) return st;
    for (int b = 0; b < batch; ++b) {
      if (ctx[b] < 0 || static_cast<long long>(ctx[b]) > static_cast<long long>(max_blocks_per_seq) * cache->block_size)
        return fail(PKV_ERR_INVALID_ARG, "context_lens[%d] = %d out of range", b, ctx[b]);
      for (int j = 0; j < (ctx[b] + cache->block_size - 1) / cache->block_size; ++j) {
        const int32_t blk = bt[static_cast<size_t>(b) * max_blocks_per_seq + j];
        if (blk < 0 || blk >= cache->num_blocks)
          return fail(PKV_ERR_INVALID_ARG, "block_tables[%d][%d] = %d outside [0, %d)", b, j, blk,
                      cache->num_blocks);
      }
    }
  }

  if ((st = encode_cache_map(&L.kmap, k_cache, cache)) != PKV_OK) return st;
  if ((st = encode_cache_map(&L.vmap, v_cache, cache)) != PKV_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  L.q = q;
  L.out = out;
  L.block_tables = block_tables;
  L.context_lens = context_lens;
  const size_t scale_off = static_cast<size_t>(slot) * cache->num_blocks * cache->num_kv_heads *
                           (cache->dtype == PKV_KV_INT8 ? 2 : 1);
  L.k_scale = fp8 ? k_scale + scale_off : nullptr;
  L.v_scale = fp8 ? v_scale + scale_off : nullptr;
  L.work_counter = reinterpret_cast<int32_t*>(ws + wl.counter);
  L.unit_start = reinterpret_cast<int32_t*>(ws + wl.unit_start);
  L.ctx_eff = reinterpret_cast<int32_t*>(ws + wl.ctx_eff);
  L.part_seq = reinterpret_cast<int32_t*>(ws + wl.part_seq);
  L.arrive = reinterpret_cast<int32_t*>(ws + wl.arrive);
  L.part_ml = reinterpret_cast<float*>(ws + wl.part_ml);
  L.part_o = reinterpret_cast<float*>(ws + wl.part_o);
  if (tree != nullptr) {
    L.tree_mask = tree->mask;
    L.node_counts = tree->node_counts;
    L.tree_stride = tree->tree_batch == 1 ? 0 : num_query_tokens * L.tree_words;
    L.poison = reinterpret_cast<uint32_t*>(ws + wl.poison);
    L.v_cache = static_cast<const uint8_t*>(v_cache) + static_cast<size_t>(slot) * cache->num_blocks * cache->num_kv_heads *
                                                           cache->block_size * cache->head_dim * (fp8 ? 1 : 2);
  }
  if (L.tree_tc) {
    if (cache->dtype == PKV_KV_BF16 && (st = encode_query_map(&L.qmap, q, batch, L.T, L.Hq, L.D, L.G, L.Tt)) != PKV_OK) return st;
  } else if (L.tc && !L.tc2 && L.pmax > 1 &&
      (st = encode_partial_map(&L.pmap, L.part_o, batch, L.T, L.Hq, L.pmax, L.D, L.G, L.Tt)) != PKV_OK)
    return st;
  if (L.tc && !L.tc2 && !L.tree_tc && (st = encode_output_map(&L.omap, out, batch, L.T, L.Hq, L.D, L.G, L.Tt)) != PKV_OK)
    return st;
  if (L.tc2 && (st = encode_query_map(&L.qmap, q, batch, L.T, L.Hq, L.D, L.G, L.Tt)) != PKV_OK) return st;
  L.err = dev->err_word;
  L.row_base = static_cast<int>(static_cast<long long>(slot) * cache->num_blocks * cache->num_kv_heads *
                                cache->block_size);
  L.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  L.stream = s;
  if (opts != nullptr) {
    L.ev_start = static_cast<cudaEvent_t>(opts->event_decode_start);
    L.ev_end = static_cast<cudaEvent_t>(opts->event_decode_end);
  }
  pkv::AppendArgs app{};
  if (req != nullptr && req->num_tokens > 0) {
    if ((st = prepare_append(cache, slot, req->k, req->v, req->slot_mapping, req->num_tokens,
                             const_cast<void*>(k_cache), const_cast<void*>(v_cache), k_scale, v_scale, s,
                             dev, &app)) != PKV_OK)
      return st;
    L.append = &app;
    L.append_kind = cache->dtype;
  }
  int launched = 0;
  cudaError_t e = L.tree_tc ? pkv::launch_tree_attend(L, ws, &launched) : pkv::launch_decode(L, &launched);
  if (e != cudaSuccess) return cuda_fail(e, "paged_decode launch");
  return PKV_OK;
}

extern "C" {

pkv_status pkv_paged_decode_multi(const pkv_cache_desc* cache, const void* q, int32_t batch,
                                  int32_t num_query_tokens, int32_t num_q_heads, const void* k_cache,
                                  const void* v_cache, const float* k_scale, const float* v_scale,
                                  const int32_t* block_tables, int32_t max_blocks_per_seq,
                                  const int32_t* context_lens, const int32_t* kv_group_ptr,
                                  int32_t num_layers, int32_t layer, float scale, void* out,
                                  void* workspace, size_t workspace_bytes,
                                  const pkv_decode_opts* opts, void* stream) {
  return decode_call(cache, q, batch, num_query_tokens, num_q_heads, k_cache, v_cache, k_scale, v_scale,
                     block_tables, max_blocks_per_seq, context_lens, kv_group_ptr, num_layers, layer, scale,
                     out, workspace, workspace_bytes, opts, stream, nullptr);
}

pkv_status pkv_append_and_decode(const pkv_cache_desc* cache, const void* k_new, const void* v_new,
                                 const int64_t* slot_mapping, int32_t num_new_tokens, const void* q,
                                 int32_t batch, int32_t num_query_tokens, int32_t num_q_heads,
                                 void* k_cache, void* v_cache, const float* k_scale, const float* v_scale,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* context_lens, const int32_t* kv_group_ptr,
                                 int32_t num_layers, int32_t layer, float scale, void* out,
                                 void* workspace, size_t workspace_bytes, const pkv_decode_opts* opts,
                                 void* stream) {
  if (num_new_tokens < 0) return fail(PKV_ERR_INVALID_ARG, "num_new_tokens %d < 0", num_new_tokens);
  const AppendRequest req{k_new, v_new, slot_mapping, num_new_tokens};
  return decode_call(cache, q, batch, num_query_tokens, num_q_heads, k_cache, v_cache, k_scale, v_scale,
                     block_tables, max_blocks_per_seq, context_lens, kv_group_ptr, num_layers, layer, scale,
                     out, workspace, workspace_bytes, opts, stream, &req);
}

pkv_status pkv_paged_decode(const pkv_cache_desc* cache, const void* q, int32_t batch,
                            int32_t num_q_heads, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale,
                            const int32_t* block_tables, int32_t max_blocks_per_seq,
                            const int32_t* context_lens, const int32_t* kv_group_ptr,
                            int32_t num_layers, int32_t layer, float scale, void* out,
                            void* workspace, size_t workspace_bytes, const pkv_decode_opts* opts,
                            void* stream) {
  return pkv_paged_decode_multi(cache, q, batch, 1, num_q_heads, k_cache, v_cache, k_scale, v_scale,
                                block_tables, max_blocks_per_seq, context_lens, kv_group_ptr,
                                num_layers, layer, scale, out, workspace, workspace_bytes, opts,
                                stream);
}

pkv_status pkv_paged_decode_tree(const pkv_cache_desc* cache, const void* q, int32_t batch,
                                 int32_t num_query_tokens, int32_t num_q_heads, const void* k_cache,
                                 const void* v_cache, const float* k_scale, const float* v_scale,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* context_lens, const uint32_t* tree_mask,
                                 int32_t tree_batch, const int32_t* node_counts,
                                 const int32_t* kv_group_ptr, int32_t num_layers, int32_t layer,
                                 float scale, void* out, void* workspace, size_t workspace_bytes,
                                 const pkv_decode_opts* opts, void* stream) {
  const TreeRequest tree{tree_mask, tree_batch, node_counts};
  return decode_call(cache, q, batch, num_query_tokens, num_q_heads, k_cache, v_cache, k_scale, v_scale,
                     block_tables, max_blocks_per_seq, context_lens, kv_group_ptr, num_layers, layer, scale,
                     out, workspace, workspace_bytes, opts, stream, nullptr, &tree);
}

pkv_status pkv_paged_decode_packed(const pkv_cache_desc* cache, const void* q, int32_t num_rows, int32_t batch,
                                   int32_t max_query_tokens, int32_t num_q_heads, const void* k_cache,
                                   const void* v_cache, const float* k_scale, const float* v_scale,
                                   const int32_t* block_tables, int32_t max_blocks_per_seq,
                                   const int32_t* context_lens, const int32_t* query_starts,
                                   const int32_t* kv_group_ptr, int32_t num_layers, int32_t layer, float scale,
                                   void* out, void* workspace, size_t workspace_bytes,
                                   const pkv_decode_opts* opts, void* stream) {
  pkv::DecodeLaunch L;
  pkv_status st = resolve_packed(cache, num_rows, batch, max_query_tokens, num_q_heads, max_blocks_per_seq, opts, &L);
  if (st != PKV_OK) return st;
  if (kv_group_ptr == nullptr || num_layers < 1 || layer < 0 || layer >= num_layers)
    return fail(PKV_ERR_INVALID_ARG, "layer %d / num_layers %d / kv_group_ptr", layer, num_layers);
  const int32_t slot = kv_group_ptr[layer];
  if (slot < 0 || slot >= cache->num_slots)
    return fail(PKV_ERR_INVALID_ARG, "kv_group_ptr[%d] = %d outside [0, %d)", layer, slot, cache->num_slots);
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale is not finite");
  if (batch == 0 || num_rows == 0) return PKV_OK;
  const bool fp8 = cache->dtype != PKV_KV_BF16;  // one-byte elements (E4M3 or INT8)
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_starts || !out)
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (fp8 && (!k_scale || !v_scale)) return fail(PKV_ERR_INVALID_ARG, "E4M3 and INT8 caches need k_scale and v_scale");
  if (fp8 && !scales_aligned(cache->dtype, k_scale, v_scale))
    return fail(PKV_ERR_ALIGNMENT, "k_scale and v_scale must be 4-byte (E4M3) or 8-byte (INT8) aligned");
  if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace))
    return fail(PKV_ERR_ALIGNMENT, "q, out, caches and workspace must be 16-byte aligned");
  if (!aligned4({block_tables, context_lens, query_starts}))
    return fail(PKV_ERR_ALIGNMENT, "block_tables, context_lens and query_starts must be 4-byte aligned");
  const size_t row = static_cast<size_t>(num_q_heads) * cache->head_dim * 2, lens = static_cast<size_t>(batch) * 4;
  const size_t slot_rows = static_cast<size_t>(cache->num_blocks) * cache->num_kv_heads;  // pages of a slot
  const size_t pool = cache->num_slots * slot_rows * cache->block_size * cache->head_dim * (fp8 ? 1 : 2);
  if (!disjoint({{out, num_rows * row}}, {{q, num_rows * row}, {block_tables, lens * max_blocks_per_seq}, {context_lens, lens},
                                          {query_starts, lens + 4}, {k_cache, pool}, {v_cache, pool}}))
    return fail(PKV_ERR_INVALID_ARG, "out overlaps another array");
  const size_t need = packed_total(L);
  if (workspace == nullptr || workspace_bytes < need)
    return fail(PKV_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if ((st = device_info(&dev)) != PKV_OK) return st;
  if (env_flag("PKV_VALIDATE")) {
    std::vector<int32_t> ctx, starts, bt;
    if ((st = fetch(ctx, context_lens, static_cast<size_t>(batch), s)) != PKV_OK) return st;
    if ((st = fetch(starts, query_starts, static_cast<size_t>(batch) + 1, s)) != PKV_OK) return st;
    if ((st = fetch(bt, block_tables, static_cast<size_t>(batch) * max_blocks_per_seq, s)) != PKV_OK) return st;
    for (int b = 0; b < batch; ++b) {
      if (starts[b] < 0 || starts[b + 1] < starts[b] || starts[b + 1] > num_rows || starts[b + 1] - starts[b] > L.T)
        return fail(PKV_ERR_INVALID_ARG, "query_starts[%d], [%d] = %d, %d", b, b + 1, starts[b], starts[b + 1]);
      if (ctx[b] < 0 || static_cast<long long>(ctx[b]) > static_cast<long long>(max_blocks_per_seq) * cache->block_size)
        return fail(PKV_ERR_INVALID_ARG, "context_lens[%d] = %d out of range", b, ctx[b]);
      if (starts[b + 1] == starts[b]) continue;
      for (int j = 0; j < (ctx[b] + cache->block_size - 1) / cache->block_size; ++j) {
        const int32_t blk = bt[static_cast<size_t>(b) * max_blocks_per_seq + j];
        if (blk < 0 || blk >= cache->num_blocks)
          return fail(PKV_ERR_INVALID_ARG, "block_tables[%d][%d] = %d outside [0, %d)", b, j, blk, cache->num_blocks);
      }
    }
  }
  if ((st = encode_cache_map(&L.kmap, k_cache, cache)) != PKV_OK) return st;
  if ((st = encode_cache_map(&L.vmap, v_cache, cache)) != PKV_OK) return st;
  if (!fp8 && (st = encode_query_map(&L.qmap, q, 1, num_rows, L.Hq, L.D, L.G, L.Tt)) != PKV_OK) return st;
  L.q = q;
  L.out = out;
  L.block_tables = block_tables;
  L.context_lens = context_lens;
  L.query_starts = query_starts;
  const size_t scale_off = slot * slot_rows * (cache->dtype == PKV_KV_INT8 ? 2 : 1);
  L.k_scale = fp8 ? k_scale + scale_off : nullptr;
  L.v_scale = fp8 ? v_scale + scale_off : nullptr;
  L.v_cache = static_cast<const uint8_t*>(v_cache) + slot * slot_rows * cache->block_size * cache->head_dim * (fp8 ? 1 : 2);
  L.err = dev.err_word;
  L.row_base = static_cast<int>(static_cast<long long>(slot) * slot_rows * cache->block_size);
  L.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  L.stream = s;
  L.num_sms = dev.num_sms;
  L.tree_shares = pkv::packed_most_shares(dev.num_sms);  // (the workspace was checked for the most)
  if (opts != nullptr) {
    L.ev_start = static_cast<cudaEvent_t>(opts->event_decode_start);
    L.ev_end = static_cast<cudaEvent_t>(opts->event_decode_end);
  }
  int launched = 0;
  cudaError_t e = pkv::launch_packed_attend(L, static_cast<uint8_t*>(workspace), &launched);
  if (e != cudaSuccess) return cuda_fail(e, "paged_decode_packed launch");
  return PKV_OK;
}

pkv_status pkv_tree_masks(const int32_t* parents, const int32_t* context_lens, const int32_t* node_counts,
                          int32_t batch, int32_t num_nodes, uint32_t* mask, int32_t* positions,
                          void* stream) {
  if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (num_nodes < 1 || num_nodes > PKV_MAX_QUERY_TOKENS)
    return fail(PKV_ERR_INVALID_ARG, "num_nodes %d outside 1..%d", num_nodes, PKV_MAX_QUERY_TOKENS);
  if (batch == 0) return PKV_OK;
  if (!parents || !mask) return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned4({parents, context_lens, node_counts, mask, positions}))
    return fail(PKV_ERR_ALIGNMENT, "every array must be 4-byte aligned");
  const size_t nodes = static_cast<size_t>(batch) * num_nodes * 4, words = nodes * ((num_nodes + 31) / 32);
  const size_t lens = static_cast<size_t>(batch) * 4;
  if (!disjoint({{mask, words}, {positions, nodes}}, {{parents, nodes}, {context_lens, lens}, {node_counts, lens}}))
    return fail(PKV_ERR_INVALID_ARG, "mask and positions must not overlap other arrays");
  DeviceInfo dev;
  pkv_status st = device_info(&dev);
  if (st != PKV_OK) return st;
  const pkv::TreeMaskArgs a{parents, context_lens, node_counts, mask, positions, dev.err_word, batch, num_nodes};
  cudaError_t e = pkv::launch_tree_masks(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "tree_masks launch");
  return PKV_OK;
}

pkv_status pkv_extend_tables(int32_t batch, int32_t block_size, int32_t max_blocks_per_seq,
                             int32_t num_blocks, const int32_t* seq_lens, const int32_t* new_lens,
                             const int32_t* borrowed_counts, int32_t* block_tables,
                             const int32_t* block_counts, int32_t* new_block_counts,
                             int32_t* free_ring, int32_t* free_state, int32_t* new_free_state,
                             int32_t* context_lens, int32_t* query_starts, int64_t* slot_mapping,
                             int32_t* positions, int32_t max_tokens, void* stream) {
  if (batch < 0 || batch > PKV_MAX_TABLE_REQUESTS)
    return fail(PKV_ERR_INVALID_ARG, "batch %d outside 0..%d", batch, PKV_MAX_TABLE_REQUESTS);
  if (block_size != 16 && block_size != 32)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d (supported: 16, 32)", block_size);
  if (max_blocks_per_seq < 1 || num_blocks < 1 || max_tokens < 0)
    return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d, num_blocks %d, max_tokens %d", max_blocks_per_seq,
                num_blocks, max_tokens);
  if (static_cast<long long>(batch) * max_blocks_per_seq >= (1LL << 31) || num_blocks >= (1 << 30) ||
      static_cast<long long>(max_blocks_per_seq) * block_size >= (1LL << 31) || max_tokens >= (1 << 30))
    return fail(PKV_ERR_UNSUPPORTED, "tables, pool or token rows too large");
  if ((batch > 0 && (!seq_lens || !new_lens || !block_tables || !block_counts || !new_block_counts || !context_lens)) ||
      !free_ring || !free_state || !new_free_state || !query_starts || (max_tokens > 0 && !slot_mapping))
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned4({seq_lens, new_lens, borrowed_counts, block_tables, block_counts, new_block_counts, free_ring, free_state,
                 new_free_state, context_lens, query_starts, positions}) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
    return fail(PKV_ERR_ALIGNMENT, "arrays must be 4-byte aligned, slot_mapping 8-byte");
  const size_t lens = static_cast<size_t>(batch) * 4, rows = static_cast<size_t>(max_tokens);
  const size_t tables = lens * max_blocks_per_seq, ring = static_cast<size_t>(num_blocks) * 4;
  // the counts and the ring's state may be updated in place
  if (!disjoint({{block_tables, tables}, {free_ring, ring}, {free_state, 16}, {context_lens, lens}, {query_starts, lens + 4},
                 {slot_mapping, rows * 8}, {positions, rows * 4}, {new_block_counts, lens},
                 {new_free_state == free_state ? nullptr : new_free_state, 16}},
                {{seq_lens, lens}, {new_lens, lens}, {borrowed_counts, lens},
                 {new_block_counts == block_counts ? nullptr : block_counts, lens}}))
    return fail(PKV_ERR_INVALID_ARG, "arrays that are written overlap other arrays");
  DeviceInfo dev;
  pkv_status st = device_info(&dev);
  if (st != PKV_OK) return st;
  const pkv::ExtendArgs a{seq_lens,  new_lens,       borrowed_counts, block_tables, block_counts,
                          new_block_counts, free_ring, free_state,     new_free_state, context_lens,
                          query_starts, slot_mapping, positions,      dev.err_word, batch,
                          max_blocks_per_seq, num_blocks, block_size, max_tokens};
  cudaError_t e = pkv::launch_extend_tables(a, dev.num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "extend_tables launch");
  return PKV_OK;
}

pkv_status pkv_verify_tree(const int32_t* tokens, const int32_t* parents, const int32_t* node_counts,
                           const float* target_probs, int64_t target_stride, const float* draft_probs,
                           int64_t draft_stride, int32_t batch, int32_t num_nodes, int32_t vocab,
                           const float* accept_uniforms, const float* sample_uniforms, int32_t* accept_idx,
                           int32_t* accept_counts, int32_t max_accept, int32_t* next_tokens, void* stream) {
  if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (num_nodes < 1 || num_nodes > PKV_MAX_QUERY_TOKENS || max_accept < 1 || max_accept > PKV_MAX_QUERY_TOKENS)
    return fail(PKV_ERR_INVALID_ARG, "num_nodes %d, max_accept %d outside 1..%d", num_nodes, max_accept,
                PKV_MAX_QUERY_TOKENS);
  if (vocab < 1) return fail(PKV_ERR_INVALID_ARG, "vocab %d < 1", vocab);
  if (vocab > PKV_MAX_VOCAB) return fail(PKV_ERR_UNSUPPORTED, "vocab %d (supported: up to %d)", vocab, PKV_MAX_VOCAB);
  if (target_stride < vocab || (draft_probs != nullptr && draft_stride < vocab))
    return fail(PKV_ERR_INVALID_ARG, "a row stride is below the vocabulary %d", vocab);
  const int64_t stride_max = 1LL << 40;
  if (target_stride > stride_max || (draft_probs != nullptr && draft_stride > stride_max))
    return fail(PKV_ERR_UNSUPPORTED, "a row stride is above 2^40");
  if (static_cast<long long>(batch) * num_nodes >= (1LL << 24) || static_cast<long long>(batch) * max_accept >= (1LL << 24))
    return fail(PKV_ERR_UNSUPPORTED, "batch x nodes too large");
  if (batch == 0) return PKV_OK;
  if (!tokens || !parents || !target_probs || !accept_uniforms || !sample_uniforms || !accept_idx || !accept_counts || !next_tokens)
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!aligned4({tokens, parents, node_counts, target_probs, draft_probs, accept_uniforms, sample_uniforms, accept_idx,
                 accept_counts, next_tokens}))
    return fail(PKV_ERR_ALIGNMENT, "every array must be 4-byte aligned");
  const size_t lens = static_cast<size_t>(batch) * 4, nodes = lens * num_nodes, rows = static_cast<size_t>(batch) * num_nodes - 1;
  if (!disjoint({{accept_idx, lens * max_accept}, {accept_counts, lens}, {next_tokens, lens}},
                {{tokens, nodes}, {parents, nodes}, {node_counts, lens}, {accept_uniforms, nodes}, {sample_uniforms, lens},
                 {target_probs, (rows * target_stride + vocab) * 4},
                 {draft_probs, draft_probs != nullptr ? (rows * draft_stride + vocab) * 4 : 0}}))
    return fail(PKV_ERR_INVALID_ARG, "arrays that are written overlap other arrays");
  DeviceInfo dev;
  pkv_status st = device_info(&dev);
  if (st != PKV_OK) return st;
  const pkv::VerifyArgs a{tokens, parents, node_counts, target_probs, draft_probs, accept_uniforms, sample_uniforms,
                          accept_idx, accept_counts, next_tokens, dev.err_word, target_stride, draft_stride,
                          batch, num_nodes, vocab, max_accept};
  cudaError_t e = pkv::launch_verify_tree(a, dev.num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "verify_tree launch");
  return PKV_OK;
}

// new_lens, prev_lens: both or none (pkv_compact_tokens_kept).
static pkv_status compact_call(const pkv_cache_desc* cache, const int32_t* accept_idx,
                               const int32_t* accept_counts, int32_t max_accept, int32_t batch,
                               const int32_t* context_lens, const int32_t* node_counts, int32_t num_nodes,
                               const int32_t* block_tables, int32_t max_blocks_per_seq, void* k_cache,
                               void* v_cache, const float* k_scale, const float* v_scale,
                               const int32_t* new_lens, const int32_t* prev_lens, int32_t* seq_lens,
                               void* stream) {
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch %d < 0", batch);
  if (num_nodes < 1 || num_nodes > PKV_MAX_QUERY_TOKENS || max_accept < 1 || max_accept > PKV_MAX_QUERY_TOKENS)
    return fail(PKV_ERR_INVALID_ARG, "num_nodes %d, max_accept %d outside 1..%d", num_nodes, max_accept,
                PKV_MAX_QUERY_TOKENS);
  if (max_blocks_per_seq < 1) return fail(PKV_ERR_INVALID_ARG, "max_blocks_per_seq %d < 1", max_blocks_per_seq);
  if (static_cast<long long>(max_blocks_per_seq) * cache->block_size >= (1LL << 31) ||
      static_cast<long long>(batch) * cache->num_slots >= (1LL << 31))
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_seq or batch x cache slots too large");
  if (batch == 0) return PKV_OK;
  const bool fp8 = cache->dtype != PKV_KV_BF16;  // one-byte elements (E4M3 or INT8)
  if (!accept_idx || !accept_counts || !context_lens || !block_tables || !k_cache || !v_cache || !seq_lens)
    return fail(PKV_ERR_INVALID_ARG, "NULL tensor pointer");
  if (fp8 && (!k_scale || !v_scale)) return fail(PKV_ERR_INVALID_ARG, "E4M3 and INT8 caches need k_scale and v_scale");
  if (fp8 && !scales_aligned(cache->dtype, k_scale, v_scale))
    return fail(PKV_ERR_ALIGNMENT, "k_scale and v_scale must be 4-byte (E4M3) or 8-byte (INT8) aligned");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(PKV_ERR_ALIGNMENT, "caches must be 16-byte aligned");
  if (!aligned4({accept_idx, accept_counts, context_lens, node_counts, block_tables, new_lens, prev_lens, seq_lens}))
    return fail(PKV_ERR_ALIGNMENT, "index and length arrays must be 4-byte aligned");
  const size_t lens = static_cast<size_t>(batch) * 4;
  if (!disjoint({{seq_lens, lens}}, {{accept_idx, lens * max_accept}, {accept_counts, lens}, {context_lens, lens},
                                     {node_counts, lens}, {block_tables, lens * max_blocks_per_seq}, {new_lens, lens},
                                     {prev_lens == seq_lens ? nullptr : prev_lens, lens}}))
    return fail(PKV_ERR_INVALID_ARG, "seq_lens must not overlap other arrays");
  DeviceInfo dev;
  if ((st = device_info(&dev)) != PKV_OK) return st;
  const pkv::CompactArgs a{accept_idx, accept_counts, context_lens, node_counts, block_tables, new_lens, prev_lens, seq_lens,
                           static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), fp8 ? k_scale : nullptr,
                           fp8 ? v_scale : nullptr, dev.err_word, batch, max_accept, num_nodes, max_blocks_per_seq,
                           cache->num_slots, cache->num_blocks, cache->num_kv_heads, cache->block_size, cache->head_dim};
  cudaError_t e = pkv::launch_compact_tokens(cache->dtype, a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "compact_tokens launch");
  return PKV_OK;
}

pkv_status pkv_compact_tokens(const pkv_cache_desc* cache, const int32_t* accept_idx,
                              const int32_t* accept_counts, int32_t max_accept, int32_t batch,
                              const int32_t* context_lens, const int32_t* node_counts, int32_t num_nodes,
                              const int32_t* block_tables, int32_t max_blocks_per_seq, void* k_cache,
                              void* v_cache, const float* k_scale, const float* v_scale, int32_t* seq_lens,
                              void* stream) {
  return compact_call(cache, accept_idx, accept_counts, max_accept, batch, context_lens, node_counts, num_nodes,
                      block_tables, max_blocks_per_seq, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr, seq_lens,
                      stream);
}

pkv_status pkv_compact_tokens_kept(const pkv_cache_desc* cache, const int32_t* accept_idx,
                                   const int32_t* accept_counts, int32_t max_accept, int32_t batch,
                                   const int32_t* context_lens, const int32_t* node_counts, int32_t num_nodes,
                                   const int32_t* block_tables, int32_t max_blocks_per_seq, void* k_cache,
                                   void* v_cache, const float* k_scale, const float* v_scale,
                                   const int32_t* new_lens, const int32_t* prev_seq_lens, int32_t* seq_lens,
                                   void* stream) {
  if (batch > 0 && (!new_lens || !prev_seq_lens)) return fail(PKV_ERR_INVALID_ARG, "new_lens or prev_seq_lens is NULL");
  return compact_call(cache, accept_idx, accept_counts, max_accept, batch, context_lens, node_counts, num_nodes,
                      block_tables, max_blocks_per_seq, k_cache, v_cache, k_scale, v_scale, new_lens, prev_seq_lens,
                      seq_lens, stream);
}

pkv_status pkv_copy_blocks(const pkv_cache_desc* cache, const void* src_k, const void* src_v,
                           const float* src_k_scale, const float* src_v_scale, int32_t src_num_blocks,
                           void* dst_k, void* dst_v, float* dst_k_scale, float* dst_v_scale,
                           int32_t dst_num_blocks, const int32_t* block_pairs, int32_t count,
                           void* stream) {
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (count < 0 || src_num_blocks < 1 || dst_num_blocks < 1)
    return fail(PKV_ERR_INVALID_ARG, "count %d, src_num_blocks %d, dst_num_blocks %d", count,
                src_num_blocks, dst_num_blocks);
  if (count == 0) return PKV_OK;
  const bool fp8 = cache->dtype != PKV_KV_BF16;  // one-byte elements (E4M3 or INT8)
  if (!src_k || !src_v || !dst_k || !dst_v || !block_pairs)
    return fail(PKV_ERR_INVALID_ARG, "NULL pointer");
  if (fp8 && (!src_k_scale || !src_v_scale || !dst_k_scale || !dst_v_scale))
    return fail(PKV_ERR_INVALID_ARG, "E4M3 and INT8 pools need source and destination scales");
  if (fp8 && (!scales_aligned(cache->dtype, src_k_scale, src_v_scale) ||
              !scales_aligned(cache->dtype, dst_k_scale, dst_v_scale)))
    return fail(PKV_ERR_ALIGNMENT, "scales must be 4-byte (E4M3) or 8-byte (INT8) aligned");
  if (!aligned16(src_k) || !aligned16(src_v) || !aligned16(dst_k) || !aligned16(dst_v))
    return fail(PKV_ERR_ALIGNMENT, "pools must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_pairs) & 3u) != 0)
    return fail(PKV_ERR_ALIGNMENT, "block_pairs must be 4-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo dev_info;
  const DeviceInfo* dev = &dev_info;
  if ((st = device_info(&dev_info)) != PKV_OK) return st;
  if (env_flag("PKV_VALIDATE")) {
    std::vector<int32_t> pr;
    if ((st = fetch(pr, block_pairs, static_cast<size_t>(count) * 2, s)) != PKV_OK) return st;
    std::vector<int32_t> dsts;
    for (int i = 0; i < count; ++i) {
      if (pr[2 * i] < 0 || pr[2 * i] >= src_num_blocks || pr[2 * i + 1] < 0 || pr[2 * i + 1] >= dst_num_blocks)
        return fail(PKV_ERR_INVALID_ARG, "block_pairs[%d] = (%d, %d) out of range", i, pr[2 * i], pr[2 * i + 1]);
      dsts.push_back(pr[2 * i + 1]);
    }
    std::sort(dsts.begin(), dsts.end());
    if (std::adjacent_find(dsts.begin(), dsts.end()) != dsts.end())
      return fail(PKV_ERR_INVALID_ARG, "block_pairs has a repeated destination");
  }
  const int64_t block_bytes = static_cast<int64_t>(cache->num_kv_heads) * cache->block_size *
                              cache->head_dim * (fp8 ? 1 : 2);
  cudaError_t e = pkv::launch_copy_blocks(src_k, src_v, fp8 ? src_k_scale : nullptr,
                                          fp8 ? src_v_scale : nullptr, src_num_blocks, dst_k, dst_v,
                                          fp8 ? dst_k_scale : nullptr, fp8 ? dst_v_scale : nullptr,
                                          dst_num_blocks, block_pairs, count, block_bytes,
                                          cache->num_kv_heads * (cache->dtype == PKV_KV_INT8 ? 2 : 1),
                                          dev->num_sms, dev->err_word, s);
  if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
  return PKV_OK;
}

pkv_status pkv_read_probe(const void* data, size_t bytes, uint64_t* sum, void* stream) {
  if (bytes == 0) return PKV_OK;  // nothing to read, nothing launched
  if (data == nullptr || sum == nullptr) return fail(PKV_ERR_INVALID_ARG, "data or sum is NULL");
  if (bytes % 16 != 0) return fail(PKV_ERR_INVALID_ARG, "bytes %zu is not a multiple of 16", bytes);
  if (reinterpret_cast<uintptr_t>(data) % 16 != 0 || reinterpret_cast<uintptr_t>(sum) % 8 != 0)
    return fail(PKV_ERR_ALIGNMENT, "data must be 16-byte and sum 8-byte aligned");
  DeviceInfo dev_info;
  const DeviceInfo* dev = &dev_info;
  pkv_status st = device_info(&dev_info);
  if (st != PKV_OK) return st;
  cudaError_t e = pkv::launch_read_probe(data, bytes, reinterpret_cast<unsigned long long*>(sum), dev->num_sms,
                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "read probe launch");
  return PKV_OK;
}

pkv_status pkv_read_device_error(uint32_t* flags, void* stream) {
  if (flags == nullptr) return fail(PKV_ERR_INVALID_ARG, "flags is NULL");
  DeviceInfo dev_info;
  const DeviceInfo* dev = &dev_info;
  pkv_status st = device_info(&dev_info);
  if (st != PKV_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned host = 0;
  cudaError_t e = cudaMemcpyAsync(&host, dev->err_word, sizeof host, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(dev->err_word, 0, sizeof host, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
  *flags = host;
  if (host != 0) {
    set_error("device error word 0x%x", host);
    return PKV_ERR_DEVICE_INDEX;
  }
  return PKV_OK;
}

}  // extern "C"
