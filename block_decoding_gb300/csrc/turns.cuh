// Frequencies as fractions of a turn. Host code only: a test compiles it by itself.
#pragma once

#include <math.h>

namespace dllm {

// freq / 2 pi modulo 1 as a 64-bit fraction, within one unit: the product with
// 1 / 2 pi in two parts, so that its error is that of the last bit kept. Of the
// size, for what is left of a whole turn is exact from 0 up only (below, -2^-60 + 1
// is 1); a fraction's negative is exact.
inline unsigned long long fraction_of_turn(double freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1 / 2 pi = kHi + kLo
  const double size = fabs(freq), hi = size * kHi, lo = fma(size, kHi, -hi) + size * kLo;
  const double whole = hi - floor(hi);                                        // exact, in [0, 1)
  // (1 - 2^-53 is the most it can be; the sum wraps around a turn)
  const unsigned long long turns =
      static_cast<unsigned long long>(whole * 0x1p64) + static_cast<unsigned long long>(llrint(lo * 0x1p64));
  return freq < 0 ? 0ull - turns : turns;
}

}  // namespace dllm
