// Whose rows the attention of packed rows serves, as its planner decides (no CUDA).
#include <cstdint>

#include "packed_plan.cuh"

using namespace pkv;

extern "C" {

// served[b]: whether sequence b's rows are; owner[row]: the sequence that the scan
// of rows takes the row for, -1 where it has none.
void packed_starts(const int32_t* starts, int B, int N, int T, int32_t* served, int32_t* owner) {
  int fall = B;
  for (int b = B - 1; b >= 0; --b)
    if (packed_falls(starts, b)) fall = b;
  for (int b = 0; b < B; ++b) served[b] = packed_rows_fit(starts[b], starts[b + 1], b, fall, N, T) ? 1 : 0;
  for (int row = 0; row < N; ++row) {
    const int b = packed_owner(starts, fall, row);
    owner[row] = b >= 0 && served[b] && row < starts[b + 1] ? b : -1;
  }
}
}
