// e2m1 codes and the powers of two of their groups (the 4-bit cache).
//
// A row (one token, one kv head, K or V) is d codes c_i, two a byte (element 2 i in
// bits 0-3 of byte i, 2 i + 1 in bits 4-7), and d / 32 bytes e, one for every 32
// neighbouring elements: their values are c_i * 2^(e - 127). e2m1 holds 0, 0.5, 1, 1.5,
// 2, 3, 4, 6 and their negatives. The factor is a power of two, so scaling is exact:
// a code is the nearest e2m1 value of the scaled element (one rounding, ties to even).
//   e = 0    a group of zeros: the factor reads as 0
//   e = 255  the group is not finite. One that held a NaN or an infinity is written with
//            codes of zero. The read-back takes the factor as infinity, and 0 * inf is
//            NaN; decode takes all 32 as NaN whatever their codes
// Smallest factor. 6 is the largest code and the codes next to it are 2 apart, so up to
// 7 times the factor no element is off by more than elements between 4 and 6 may be; with
// the factor twice as large it would be off as much, and all others more. So e is the
// smallest with max |x_i| <= 7 * 2^(e - 127) (not 6: groups whose largest element lies
// between 6 and 7 keep a bit more). At most 252: 6 * 2^125 is the largest finite value.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

constexpr int kFp4Group = 32;

// Byte e of a group whose largest magnitude has the fp32 bits `top`: 7 = 1.75 * 2^2, so
// e is the exponent field less 2, plus one when the fraction is above 0.75.
__device__ __forceinline__ int group_exponent(uint32_t top) {
  if (top == 0u) return 0;
  if (top >= 0x7f800000u) return 255;
  const int e = static_cast<int>(top >> 23) - 2 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, 1), 252);
}

// Eight values to codes (nearest, ties to even; magnitudes above 6 become 6), x[0] in
// bits 0-3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n"
      " .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n"
      "}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight codes to fp16 values, exactly, in order.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t codes, uint32_t (&r)[4]) {
  asm("{\n"
      " .reg .b8 b0, b1, b2, b3;\n"
      " mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      " cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      " cvt.rn.f16x2.e2m1x2 %3, b3;\n"
      "}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(codes));
}

}  // namespace pa
