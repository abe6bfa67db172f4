// The frequencies of the rotary append as it keeps them (no CUDA).
#include "rope_turns.h"

extern "C" unsigned long long rope_turns(double inv_freq) { return pkv::rope_turns(inv_freq); }
