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
//
// And the shared memory of the product of such codes (splitk_mx4_gemm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk_device.cuh"
#include "splitk_internal.h"

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

// ---------------------------------------------------------------- the product's shared memory
constexpr int kTileK = 256;                          // codes of a K tile: 128 bytes
constexpr int kMxStages = 4;                         // of the ring, at most
// K tiles of a stage: a stage's wait and commit take the issuing warp ~230 clocks and its
// scales a scale warp ~400, the MMAs of one tile 288 to 512 (1x500x16384 7.3 us with one,
// 6.7 with two; 16x4096x7168 7.5, 7.4; 7x2080x256 3.7, 3.8).  Each tile's
// place is free for the next copies by itself (with whole stages, the copies came too late:
// 2048x18432x7168 93 us, so 90; 1000x7168x16384 54, 51).
constexpr int kSub = 2;
constexpr uint32_t kCodesA = kMmaM * (kTileK / 2);   // 16 KiB
constexpr uint32_t kScaleAtom = 512;                 // 128 rows x 4 scales
constexpr int kGroup = 4;                            // K tiles whose scales the scale warps exchange at once
constexpr uint32_t kMxBarBytes = 512;

// (of the half of the tokens that a CTA brings)
__host__ __device__ constexpr uint32_t codes_b(int tok) { return (uint32_t)tok / 2 * (kTileK / 2); }
__host__ __device__ constexpr int groups_b(int tok) { return (tok + 127) / 128; }     // of 128 tokens
__host__ __device__ constexpr uint32_t scales_of(int tok) { return 2u * kScaleAtom * (1u + groups_b(tok)); }
__host__ __device__ constexpr uint32_t stage_bytes(int tok) { return kSub * (kCodesA + codes_b(tok)); }

// A CTA's shared memory: codes of A, codes of B, scales, barriers.  A share of split K
// leaves its sums from the start on (tokens of 128 f32), over what its MMAs have read, while
// others still wait on the barriers: they lie behind the longer of both.  (256 tokens'
// sums pass a ring of one stage, 128 KiB and 88.)
__host__ __device__ constexpr uint32_t mx_ring_bytes(int tok, int stages) {
  return (uint32_t)stages * stage_bytes(tok) + 2u * kGroup * scales_of(tok);
}
__host__ __device__ constexpr uint32_t mx_sum_bytes(int tok, int split) { return split > 1 ? (uint32_t)tok * kMmaM * 4u : 0u; }
__host__ __device__ constexpr uint32_t mx_bars_at(int tok, int stages, int split) {
  return mx_ring_bytes(tok, stages) > mx_sum_bytes(tok, split) ? mx_ring_bytes(tok, stages) : mx_sum_bytes(tok, split);
}

}  // namespace splitk
