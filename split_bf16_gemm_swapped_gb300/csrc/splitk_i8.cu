// splitk_gemm_i8(): argument checks and the choice of kernel for the product
// of 8-bit codes.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"
#include "splitk_i8.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

// Few tokens stream through registers; from 33 on the tensor core's rate for
// f16 (mma.sync: 604 TFLOP/s measured) would bound the stream.  Tiles of up to
// 128 tokens; K is split while that gives more SMs a tile, two K tiles a rank
// at least.
I8Plan plan_i8(int M, int N, int K, int L, const DeviceSize& dev) {
  if (M <= 32) return I8Plan{false, M <= 8 ? 8 : M <= 16 ? 16 : 32, 1, 0};
  I8Plan pl{true, M <= 64 ? 64 : 128, 1, 4};
  const long long tiles = (long long)((M + pl.tokens - 1) / pl.tokens) * ((N + 127) / 128) * L;
  const int k_tiles = (K + 127) / 128;
  while (pl.split < 8 && tiles * pl.split * 2 <= dev.num_sms && k_tiles / (pl.split * 2) >= 2) pl.split *= 2;
  return pl;
}

}  // namespace

}  // namespace splitk

using namespace splitk;

extern "C" {

SPLITK_API int splitk_gemm_i8(const void* a_q, const float* a_scale, const void* b_q, const float* b_scale,
                              const void* bias, void* c, int c_type, int M, int N, int K, int L,
                              splitk_stream_t stream) {
  if (!a_q || !a_scale || !b_q || !b_scale || !c) return SPLITK_ERR_NULL;
  if (c_type != SPLITK_DTYPE_BF16 && c_type != SPLITK_DTYPE_F32) return SPLITK_ERR_INVALID_ARGUMENT;
  if (M < 1 || N < 1 || K < 1 || L < 1 || K % 16 != 0 || L > 65535 || N > 65535 * 16 || M > 65535 * 32 ||
      K > (1 << 30)) {
    return SPLITK_ERR_INVALID_SHAPE;
  }
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(bias, 2) ||
      !aligned(c, c_type == SPLITK_DTYPE_F32 ? 4u : 2u)) {
    return SPLITK_ERR_MISALIGNED;
  }
  DeviceSize dev;
  int rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  const I8Params p{static_cast<const int8_t*>(a_q), static_cast<const int8_t*>(b_q), a_scale, b_scale,
                   static_cast<const uint16_t*>(bias), c, c_type == SPLITK_DTYPE_F32, M, N, K, L};
  const I8Plan plan = plan_i8(M, N, K, L, dev);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(plan.tile ? launch_i8_tile(p, plan, wait_limit_ns(), s) : launch_i8_stream(p, plan, s));
}

}  // extern "C"
