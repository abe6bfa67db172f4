// Frequencies of the rotary append as fractions of a turn (without CUDA, so that
// a host test can check them).
#pragma once

#include <cmath>
#include <cstdint>

namespace pkv {

// x turns modulo one, in 2^-64, to one unit.  (By size and sign: 1 - a small x
// would lose the bits of x.)
inline uint64_t turns_part(double x) {
  const double a = std::fabs(x), part = a - std::floor(a);  // exact
  const double units = part * 18446744073709551616.0;       // (x 2^64, below it)
  const uint64_t t = units < 9007199254740992.0 ? static_cast<uint64_t>(units + 0.5) : static_cast<uint64_t>(units);
  return x < 0 ? 0 - t : t;
}

// Turns per position of a frequency in radians, modulo one, in 2^-64.  The
// position multiplies what this is off by, so the quotient has two parts: with
// 1 / 2 pi in two doubles and the first product's rounding taken back, it is right
// to two units up to 2^40 radians (one double alone: 2^-24.5 of half a turn at
// the last int32 position for one radian).
inline uint64_t rope_turns(double inv_freq) {
  constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
  const double high = inv_freq * kHigh;
  const double low = std::fma(inv_freq, kLow, std::fma(inv_freq, kHigh, -high));
  return turns_part(high) + turns_part(low);
}

}  // namespace pkv
