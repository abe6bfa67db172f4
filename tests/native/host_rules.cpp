// Rules that kernels share with the host, for the CPU tests (no CUDA).
#include "stage_ring.h"

extern "C" {
int stage_bars(void) { return pkv::kStageBars; }
unsigned stage_bar(unsigned n) { return pkv::stage_bar(n); }
unsigned stage_parity(unsigned n) { return pkv::stage_parity(n); }
}
