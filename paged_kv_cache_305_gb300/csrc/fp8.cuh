// e4m3 codes and their power-of-two row factors (the 8-bit cache).
//
// A row (one token, one kv head, K or V) is d codes c_i and one biased
// exponent byte e: its values are c_i * 2^(e - 127). The factor is a power of
// two so that scaling is exact in both directions: a code is the nearest e4m3
// value of the scaled element (one rounding, ties to even), a read is exact
// unless the 16-bit type it is rounded to has fewer bits or less range. e4m3
// keeps four significant bits over 2^-6 .. 448, so a factor that is up to
// twice the smallest possible one costs range at the small end, no bits.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

// Byte e of a row whose largest finite magnitude is `top` (>= 0): the smallest
// e in [1, 254] with top <= 448 * 2^(e - 127). 448 = 1.75 * 2^8, so e is the
// exponent field of `top` less 8, plus one when its fraction is above 0.75.
__device__ __forceinline__ int row_exponent(float top) {
  const int b = __float_as_int(top);
  const int e = (b >> 23) - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(max(e, 1), 254);
}

// 2^(e - 127) for e in [1, 254] (e = 0 gives 0, e = 255 infinity).
__device__ __forceinline__ float exponent_factor(int e) { return __int_as_float(e << 23); }

// Two values to e4m3 codes (nearest, ties to even; NaN stays NaN; magnitudes
// above 448 saturate, which scaled finite elements never reach); lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes (bits 0-7 and 8-15) to fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

}  // namespace pa
