// Block tables, slot mapping and positions of a step's new tokens, on the GPU.
//
// Request b has s_b cached tokens in h_b blocks and adds a_b.  It needs
//   need_b = max(0, ceil((s_b + a_b) / bs) - h_b)
// more blocks, which come off the head of a ring of free block ids in request
// order: the first at ring position head + sum_{b' < b} need_b'.  Requests that
// end give their blocks back behind the ring's tail.  Both are prefix sums, so
// which block goes where depends on the inputs alone, not on timing, and no id
// is handed out by an atomic.  Token i of request b is at position p = s_b + i,
// in slot table[p / bs] * bs + p % bs.
//
// One launch.  Every CTA makes the three prefix sums (token rows, blocks
// needed, blocks given back) over all requests for itself, in shared memory:
// that costs each CTA B reads of three arrays out of L2 (3 KB for 256
// requests), less than a grid-wide barrier or a second launch.  Then
// the CTAs share the token rows, the taken and the returned blocks, each found
// by binary search in its prefix sums.  A request whose blocks to give back
// hold an id that is no block gives none back, which the other requests' places
// in the ring depend on: so the CTAs that return blocks look at all of those
// ids first.  They are the last ones, which have the fewest token rows (all
// CTAs, before the token rows: 1 us more for the prompts below).  Counts and the ring's head may be
// updated in place although every CTA reads them: the CTA that arrives last,
// when all others have read theirs, writes them (with one CTA, or arrays apart,
// nobody waits).
//
// Bound by latency: 256 requests of 8 to 32 new tokens, of which a tenth end
// with some 130 blocks each, take 9 to 10 us with the host's call, the longer of
// the two; 48 prompts of up to 24,000 tokens (570,000 rows, 6.9 MB written) 10.6
// us.  There a thread takes runs of
// four rows, which mostly share their request and block: one search, one table
// entry, wide stores (a row per thread at a time: 15 us).
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kExtThreads = 512;
constexpr int kExtRun = 4;   // token rows of a thread where there are many
constexpr int kExtLook = 8;  // returned blocks that a thread looks at together

struct ExtRequest {
  int seq, add, held, need, gone, borrowed;
  bool valid, done;
};

__device__ __forceinline__ ExtRequest ext_request(const ExtendArgs& a, int b) {
  ExtRequest r;
  r.seq = a.seq_lens[b];
  r.held = a.counts_in[b];
  const int fresh = a.new_lens[b];
  r.done = fresh == -1;
  r.add = max(fresh, 0);
  const long long total = static_cast<long long>(r.seq) + r.add;
  r.valid = r.held >= 0 && r.held <= a.MB &&
            (r.done || (fresh >= 0 && r.seq >= 0 && total <= static_cast<long long>(a.MB) * a.bs &&
                        r.seq <= static_cast<long long>(r.held) * a.bs));
  r.need = r.valid && !r.done ? max(0, static_cast<int>((total + a.bs - 1) / a.bs) - r.held) : 0;
  r.borrowed = a.borrowed != nullptr ? min(max(a.borrowed[b], 0), max(r.held, 0)) : 0;
  r.gone = r.valid && r.done ? r.held - r.borrowed : 0;
  return r;
}

// The entry b of prefix sums pre[0 .. n] with pre[b] <= i < pre[b + 1].
__device__ __forceinline__ int ext_find(const int* pre, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] > i) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Block number k of those given back, rel[b] <= k < rel[b + 1], is at [k].
__device__ __forceinline__ const int32_t* ext_given_back(const ExtendArgs& a, const int* rel, int b) {
  return a.block_tables + static_cast<size_t>(b) * a.MB + (a.borrowed != nullptr ? max(a.borrowed[b], 0) : 0) - rel[b];
}

// Marks the ended requests with an id that is no block among those to give back,
// and takes them out of rel.  Returns whether there are any.  Whole CTA.
__device__ __forceinline__ bool ext_faults(const ExtendArgs& a, int* rel, uint32_t* faulty) {
  const int B = a.B, tid = threadIdx.x, lane = tid & 31, total = rel[B];
  for (int i = tid; i < (B + 31) / 32; i += kExtThreads) faulty[i] = 0u;
  __syncthreads();
  bool wrong = false;
  // runs of up to kExtLook blocks a thread, which mostly are one request's:
  // one search, and the loads in flight together
  const int look = min(kExtLook, (total + kExtThreads - 1) / kExtThreads);
  for (int k0 = tid * look; k0 < total; k0 += kExtThreads * look) {
    int id[kExtLook], of[kExtLook];
    int b = 0, end = 0;
    const int32_t* row = nullptr;
#pragma unroll
    for (int u = 0; u < kExtLook; ++u) {
      id[u] = 0;
      const int k = k0 + u;
      if (u >= look || k >= total) continue;
      if (k >= end) {
        b = ext_find(rel, B, k);
        end = rel[b + 1];
        row = ext_given_back(a, rel, b);
      }
      id[u] = row[k];
      of[u] = b;
    }
#pragma unroll
    for (int u = 0; u < kExtLook; ++u)
      if (static_cast<uint32_t>(id[u]) >= static_cast<uint32_t>(a.NB)) {
        wrong = true;
        atomicOr(&faulty[of[u] >> 5], 1u << (of[u] & 31));
      }
  }
  if (!__syncthreads_or(wrong)) return false;
  if (tid < 32) {
    int carry = 0;
    for (int c = 0; c <= B; c += 32) {
      const int b = c + lane;
      const int gone = b < B && !((faulty[b >> 5] >> (b & 31)) & 1u) ? rel[b + 1] - rel[b] : 0;
      int x = gone;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      __syncwarp();  // (the next 32 read no entry that is written here)
      if (b <= B) rel[b] = carry + x - gone;
      carry += __shfl_sync(kFull, x, 31);
    }
  }
  __syncthreads();
  return true;
}
__device__ __noinline__ bool ext_faults_again(const ExtendArgs& a, int* rel, uint32_t* faulty) { return ext_faults(a, rel, faulty); }

__global__ void __launch_bounds__(kExtThreads) extend_tables_kernel(const ExtendArgs a) {
  extern __shared__ int sm_ext[];
  __shared__ long long warp_tok[kExtThreads / 32];
  __shared__ int warp_need[kExtThreads / 32], warp_gone[kExtThreads / 32];
  __shared__ int last_s, faults_s, taken_s;
  const int B = a.B, N = a.N;
  const uint32_t NB = static_cast<uint32_t>(a.NB);
  int* tok = sm_ext;         // [B + 1] first token row of each request, at most N
  int* blk = tok + B + 1;    // [B + 1] blocks that the requests before need
  int* rel = blk + B + 1;    // [B + 1] blocks that the requests before give back
  uint32_t* faulty = reinterpret_cast<uint32_t*>(rel + B + 1);  // [B bits] ended requests with ids that are no blocks
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int head = a.state_in[0], free_blocks = a.state_in[1];

  // prefix sums: a run of consecutive requests per thread, one scan over the threads
  const int per = (B + kExtThreads - 1) / kExtThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long st = 0;  // token rows: 64 bits, the lengths are not trusted
  int sn = 0, sg = 0;
  for (int b = b0; b < b1; ++b) {
    const ExtRequest r = ext_request(a, b);
    st += r.add;
    sn += r.need;
    sg += r.gone;
  }
  long long xt = st;
  int xn = sn, xg = sg;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long yt = __shfl_up_sync(kFull, xt, o);
    const int yn = __shfl_up_sync(kFull, xn, o), yg = __shfl_up_sync(kFull, xg, o);
    if (lane >= o) {
      xt += yt;
      xn += yn;
      xg += yg;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = xt;
    warp_need[warp] = xn;
    warp_gone[warp] = xg;
  }
  if (tid == 0) taken_s = 0;
  __syncthreads();
  xt -= st;
  xn -= sn;
  xg -= sg;
  for (int w = 0; w < warp; ++w) {
    xt += warp_tok[w];
    xn += warp_need[w];
    xg += warp_gone[w];
  }
  for (int b = b0; b < b1; ++b) {
    const ExtRequest r = ext_request(a, b);
    tok[b] = static_cast<int>(min(xt, static_cast<long long>(N)));
    blk[b] = xn;
    rel[b] = xg;
    xt += r.add;
    xn += r.need;
    xg += r.gone;
  }
  // the thread with the last request (or the first thread without any)
  if (b1 == B && (b0 < B || (B == 0 && tid == 0))) {
    tok[B] = static_cast<int>(min(xt, static_cast<long long>(N)));
    blk[B] = xn;
    rel[B] = xg;
  }
  __syncthreads();

  const bool pool_ok = head >= 0 && head < a.NB && free_blocks >= 0 &&
                       static_cast<long long>(free_blocks) + rel[B] <= a.NB;
  auto ring_at = [&](int k) -> uint32_t {  // position head + k, k < 2 NB
    uint32_t p = static_cast<uint32_t>(head) + static_cast<uint32_t>(k);
    if (p >= NB) p -= NB;
    if (p >= NB) p -= NB;
    return p;
  };
  auto rows_fit = [&](int b, const ExtRequest& r) { return tok[b + 1] - tok[b] == r.add; };
  // Granted requests with blocks to take come before all that are refused (a
  // request that needs blocks adds rows, and both sums only grow), so the
  // granted blocks are the first of the ring.
  auto granted = [&](int b, const ExtRequest& r) {
    return pool_ok && r.valid && !r.done && rows_fit(b, r) && (r.need == 0 || blk[b] + r.need <= free_blocks);
  };
  unsigned err = 0;
  const int first = blockIdx.x * kExtThreads + tid, stride = gridDim.x * kExtThreads;

  // token rows: one per thread, or runs of kExtRun where there are many, which
  // mostly share their request and their block
  const int run = N > stride ? kExtRun : 1;
  const bool vec = run == kExtRun && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.positions) & 15) == 0;
  for (long long i0 = static_cast<long long>(first) * run; i0 < N; i0 += static_cast<long long>(stride) * run) {
    long long slot[kExtRun];
    int pos[kExtRun];
    int b = -1, b_end = 0, block = -1, id = 0;
    bool ok = false;
    ExtRequest r{};
#pragma unroll
    for (int u = 0; u < kExtRun; ++u) {
      slot[u] = -1;
      pos[u] = 0;
      if (u >= run || i0 + u >= tok[B]) continue;
      const int i = static_cast<int>(i0 + u);
      if (b < 0 || i >= b_end) {
        b = ext_find(tok, B, i);
        b_end = tok[b + 1];
        r = ext_request(a, b);
        ok = granted(b, r);
        block = -1;
      }
      if (!ok) continue;
      const int p = r.seq + (i - tok[b]);
      const int j = p / a.bs;
      if (j != block) {
        block = j;
        id = j < r.held ? a.block_tables[static_cast<size_t>(b) * a.MB + j] : a.ring[ring_at(blk[b] + j - r.held)];
      }
      if (static_cast<uint32_t>(id) < NB) {
        slot[u] = static_cast<long long>(id) * a.bs + (p - j * a.bs);
        pos[u] = p;
      } else {
        err |= PKV_DEVERR_BLOCK_ID;
      }
    }
    if (vec && i0 + kExtRun <= N) {
      longlong2* s2 = reinterpret_cast<longlong2*>(a.slots + i0);
      s2[0] = make_longlong2(slot[0], slot[1]);
      s2[1] = make_longlong2(slot[2], slot[3]);
      if (a.positions != nullptr) *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int u = 0; u < kExtRun; ++u)
        if (u < run && i0 + u < N) {
          a.slots[i0 + u] = slot[u];
          if (a.positions != nullptr) a.positions[i0 + u] = pos[u];
        }
    }
  }
  // the CTAs that return blocks, from the last one on (the last one in any case)
  const int last_first = (gridDim.x - 1 - blockIdx.x) * kExtThreads;
  const bool looked = pool_ok && rel[B] > 0 && (last_first == 0 || last_first < rel[B]);
  const bool apart = a.counts_out != a.counts_in && a.state_out != a.state_in;
  bool faults = false;  // (block-uniform)
  if (pool_ok) {
    // taken blocks, into the requests' rows of the table (entries past those
    // that the token rows read)
    for (int k = first; k < min(blk[B], free_blocks); k += stride) {
      const int b = ext_find(blk, B, k);
      const ExtRequest r = ext_request(a, b);
      if (granted(b, r)) a.block_tables[static_cast<size_t>(b) * a.MB + r.held + (k - blk[b])] = a.ring[ring_at(k)];
    }
    // returned blocks, behind the free ones (places that no taken block is read
    // from); the thread's first one is on its way while the ids are looked at
    int k = last_first + tid, id = 0;
    if (k < rel[B]) id = ext_given_back(a, rel, ext_find(rel, B, k))[k];
    if (looked && ext_faults(a, rel, faulty)) {
      faults = true;
      err |= PKV_DEVERR_BLOCK_ID;
      if (tid == 0 && gridDim.x > 1 && !apart) atomicOr(reinterpret_cast<unsigned*>(a.state_in) + 3, 1u);
      if (k < rel[B]) id = ext_given_back(a, rel, ext_find(rel, B, k))[k];
    }
    for (; k < rel[B]; k += stride) {
      if (k >= stride) id = ext_given_back(a, rel, ext_find(rel, B, k))[k];
      a.ring[ring_at(free_blocks + k)] = id;
    }
  } else {
    err |= PKV_DEVERR_BLOCK_ID;
  }
  if (blockIdx.x == 0) {
    for (int b = tid; b < B; b += kExtThreads) {
      const ExtRequest r = ext_request(a, b);
      const bool ok = granted(b, r);
      a.context_lens[b] = ok ? r.seq + r.add : 0;
      a.query_starts[b] = tok[b];
      if (!r.valid) err |= PKV_DEVERR_CONTEXT_LEN;
      else if (!r.done && !rows_fit(b, r)) err |= PKV_DEVERR_SLOT;
      else if (!r.done && pool_ok && !ok) err |= PKV_DEVERR_NO_BLOCKS;
    }
    if (tid == 0) a.query_starts[B] = tok[B];
  }
  if (err) atomicOr(a.err, err);

  // Counts and the ring's state, once every CTA has read them: by the only
  // CTA, by the last one where they do not go where they came from, else by
  // the last one to arrive.
  __syncthreads();
  if (gridDim.x > 1 && !apart) {
    if (tid == 0) {
      unsigned* scratch = reinterpret_cast<unsigned*>(a.state_in) + 2;
      __threadfence();
      last_s = atomicInc(scratch, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0
      faults_s = last_s && atomicExch(scratch + 1, 0u) != 0u;
    }
    __syncthreads();
    if (!last_s) return;
    if (faults_s && !looked) faults = ext_faults_again(a, rel, faulty);
  } else if (blockIdx.x + 1 < gridDim.x) {
    return;
  }
  auto stays = [&](int b) { return faults && ((faulty[b >> 5] >> (b & 31)) & 1u) != 0u; };
  int taken = 0;
  for (int b = tid; b < B; b += kExtThreads) {
    const ExtRequest r = ext_request(a, b);
    int held = r.held;
    if (granted(b, r)) {
      held += r.need;
      if (r.need > 0) taken = max(taken, blk[b] + r.need);
    } else if (pool_ok && r.valid && r.done && !stays(b)) {
      held = 0;
    }
    a.counts_out[b] = held;
  }
  if (taken > 0) atomicMax(&taken_s, taken);
  __syncthreads();
  if (tid == 0) {
    if (a.state_out != a.state_in) a.state_out[2] = a.state_out[3] = 0;
    a.state_out[0] = pool_ok ? static_cast<int>(ring_at(taken_s)) : head;
    a.state_out[1] = pool_ok ? free_blocks - taken_s + rel[B] : free_blocks;
  }
}

cudaError_t launch_extend_tables(const ExtendArgs& a, int num_sms, cudaStream_t stream) {
  const size_t smem = sizeof(int) * (3 * (static_cast<size_t>(a.B) + 1) + (static_cast<size_t>(a.B) + 31) / 32);  // 199 KB at most
  if (smem > 48 * 1024 - 1024) {
    const cudaError_t e = cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int grid = std::max(1, std::min(num_sms, std::max((a.N + kExtThreads - 1) / kExtThreads, (a.B + 255) / 256)));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kExtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, extend_tables_kernel, a);
}

}  // namespace pkv
