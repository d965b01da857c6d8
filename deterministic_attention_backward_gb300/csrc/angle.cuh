// angle.cuh -- the angle of a rotary turn, position times frequency, in 128-bit fixed point (the
// reasons are in rope.cu).
#pragma once
#include <stdint.h>

namespace dash {

// A frequency in radians per position as a 128-bit fraction of a turn (whole turns fall off):
// f / (2 pi) as a sum of two doubles, 1 / (2 pi) being one too, good to 2^-105 of itself; each
// one's bits are moved to their place, which cuts off less than 2^-128 turns.  One double would
// leave 53 bits: 2e-7 radians at position 2^31, 6e-6 at 2^36.
using u128 = unsigned __int128;
__device__ __forceinline__ u128 fraction_of(double d) {
  const uint64_t b = (uint64_t)__double_as_longlong(d);
  const int sh = (int)((b >> 52) & 0x7FF) - 1023 + 76;  // mantissa's last bit at 2^(e-52)
  const u128 m = (b & 0xFFFFFFFFFFFFFull) | (1ull << 52);
  const u128 u = sh >= 128 ? 0 : sh >= 0 ? m << sh : sh > -64 ? m >> -sh : 0;
  return (b >> 63) ? 0 - u : u;
}
__device__ __forceinline__ u128 turns_of(double f) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double hi = f * kHi;
  return fraction_of(hi) + fraction_of(fma(f, kLo, fma(f, kHi, -hi)));
}

}  // namespace dash
