// Barriers of a tile's staged output (paged_decode_tc.cuh), apart from CUDA so
// that the host can check them.
//
// The compute warps stage the output in chunks, alternately in two buffers.
// Each warp arrives once per chunk; thread 0 stores a chunk when all have.  A
// warp does not wait for the others between two neighbouring chunks, so a
// barrier that both used could complete the first one's phase with two
// arrivals of a fast warp and none of a slow one, whose rows would be stored
// as they were before.  With a barrier per buffer, a warp's next arrival on
// the same barrier (two chunks on) comes after the chunk before has been
// stored: in a unit it waits until the buffer has been read, and the next
// unit's output needs P of every thread.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

constexpr int kStageBars = 2;

// Barrier and phase parity of the CTA's chunk number n (every unit has an even
// number of chunks).
PKV_HD uint32_t stage_bar(uint32_t n) { return n & 1u; }
PKV_HD uint32_t stage_parity(uint32_t n) { return (n >> 1) & 1u; }

}  // namespace pkv
