// Microscaled 4-bit floats (the OCP MXFP4 format): E2M1 codes, two in a byte with
// the first in the low nibble, and one E8M0 scale code for 32 consecutive ones.
//
//   scale code s stands for 2^(s - 127), 255 for NaN
//   a block of values v:  s = max(floor(log2(max|v|)) - 2, -126) + 127
//                         code = v / 2^(s - 127) rounded to the nearest of
//                         0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, at most 6
//
// The largest value is then 4 to 8 times its scale (past 6 it is cut off, as the
// format's standard scale does), the quotient is exact, and no scale leaves
// 1 .. 252.  A block that holds a NaN or an infinity has scale 255 and codes 0.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk_device.cuh"

namespace splitk {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNaN = 255u;

namespace dev {

// Eight values as eight codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, e;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, e};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}

}  // namespace dev

// The scale code of a block whose largest magnitude is `top` (f32: its exponent
// field is floor(log2) + 127, 0 below 2^-126, 255 for NaN and infinity).
__device__ __forceinline__ uint32_t mx_scale_code(float top) {
  const int e = (int)(__float_as_uint(top) >> 23);
  return e == 255 ? kMxNaN : (uint32_t)max(e - 2, 1);
}

// What multiplies a value of a block to give its quotient by the scale: exact (a
// power of two with exponent field 254 - code, 2 .. 253).  For a block without codes
// the quotients are of no use.
__device__ __forceinline__ float mx_inverse_scale(uint32_t code) { return __uint_as_float((254u - code) << 23); }

// The scale that a code stands for: 2^(code - 127), subnormal for 0, NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == kMxNaN ? 0x7FC00000u : code << 23);
}

}  // namespace splitk
