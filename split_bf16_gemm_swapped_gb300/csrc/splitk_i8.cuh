// 8-bit integer codes on the f16 tensor path.
//
// GB300's tensor cores have no fast 8-bit integer rate, but f16 holds every
// whole number up to 2048 exactly, the product of two codes is exact in the
// f32 accumulator, and so is a sum of them while its magnitude stays below
// 2^24 (any K up to 1024 whatever the codes; the partial sums of quantised
// activations and weights are far below it).  Past 2^24 the tensor cores' additions
// truncate, which for codes of one sign is a bias that grows with K (codes of
// 100..127, tiles: -9e-7 of the sum at K = 16384, -1.5e-5 at 65536, -1.4e-4 at
// 262144; streamed, whose warps each sum a share of K: 0, -3.4e-6, -5.1e-5).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk_device.cuh"

namespace splitk {
namespace dev {

__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four codes (the bytes of `w`) as two words of two f16, in order.  With the
// sign bit flipped a byte is code + 128; under the byte 0x64 it reads as the
// f16 1024 + (code + 128), and subtracting 1152 leaves the code, exactly.
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = f16x2_sub(prmt(u, 0x64646464u, 0x4140u), 0x64806480u);
  hi = f16x2_sub(prmt(u, 0x64646464u, 0x4342u), 0x64806480u);
}

}  // namespace dev

// The operands of one product (splitk_gemm_i8).
struct I8Params {
  const int8_t* a;          // weight codes [L][N][K]
  const int8_t* b;          // token codes [L][M][K]
  const float* a_scale;     // [L][N]
  const float* b_scale;     // [L][M]
  const uint16_t* bias;     // bf16 [L][N], or null
  void* c;                  // bf16 or f32 [L][M][N]
  bool c_f32;
  int M, N, K, L;
};

// The bound on its waits, and the injected failure of a test.
struct I8Waits {
  unsigned long long limit_ns;
  unsigned inject;
};

// How the tcgen05 kernel runs: tiles of 256 weight rows by `tokens`, counted
// tokens first, then rows, then batches; the first `whole` of them on one pair
// of CTAs each, the others on `split` pairs that share K.
struct I8Plan {
  int tokens;
  long long whole;
  int split;
};
cudaError_t launch_i8_stream(const I8Params& p, int num_sms, cudaStream_t stream);
cudaError_t launch_i8_tile(const I8Params& p, const I8Plan& plan, const I8Waits& waits, cudaStream_t stream);

// What one weight row's outputs share; loaded once, before the first store
// (which the compiler must take to alias it).
struct I8Channel {
  float scale, bias;
  bool has_bias;
  __device__ __forceinline__ I8Channel(const I8Params& p, int l, int n) : has_bias(p.bias != nullptr) {
    const long long at = (long long)l * p.N + n;
    scale = n < p.N ? p.a_scale[at] : 0.0f;
    bias = n < p.N && has_bias ? __uint_as_float((uint32_t)p.bias[at] << 16) : 0.0f;
  }
  // the output of the sum `v`, in f32
  __device__ __forceinline__ float result(float v, float token_scale) const {
    v = v * token_scale * scale;
    return has_bias ? v + bias : v;
  }
};

// Output (l, m, n) from its sum `v`: one rounding, from f32.
__device__ __forceinline__ void store_i8_result(const I8Params& p, int l, int m, int n, float v, float token_scale,
                                                const I8Channel& channel) {
  const float r = channel.result(v, token_scale);
  const long long at = ((long long)l * p.M + m) * p.N + n;
  if (p.c_f32) {
    static_cast<float*>(p.c)[at] = r;
  } else {
    static_cast<uint16_t*>(p.c)[at] = (uint16_t)dev::pack_bf16x2(r, 0.0f);
  }
}

}  // namespace splitk
