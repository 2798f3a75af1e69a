// The product of 8-bit codes for few tokens: the weights stream from memory
// straight into registers.
//
// A CTA owns 16 weight rows (the M side of mma.m16n8k16) and up to 32 tokens
// (its N side), and its eight warps take the 64-code chunks of K in turn, so
// that a weight row's bytes are read as whole lines.  K is the sum's index, so
// its order within a chunk is free: lane t of each group of four takes the 16
// bytes [16 t, 16 t + 16) of a row, and word j of them is the lane's share of
// the chunk's j-th product for weights and tokens alike.  Neither operand
// passes through shared memory, and a 16-byte load needs no shuffle.
//
// The warps' f32 sums are added in warp order through shared memory, so the
// result does not depend on timing.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"
#include "splitk_i8.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

constexpr int kRows = 16;            // weight rows a CTA
constexpr int kWarps = 8;
constexpr int kChunk = 64;           // codes of K a warp takes at a time

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 16 codes at `row` + k, or zeros past the row's end (K is a multiple of
// 16) or for a row that does not exist.
__device__ __forceinline__ uint4 load16(const int8_t* row, int k, int K, bool there) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (there && k < K) v = *reinterpret_cast<const uint4*>(row + k);
  return v;
}

// kTok: token columns of a CTA (8, 16 or 32).
template <int kTok>
__global__ void __launch_bounds__(32 * kWarps) i8_stream_kernel(const I8Params p) {
  constexpr int kTiles = kTok / 8;
  __shared__ float s_part[kWarps][kRows][kTok + 1];
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = (int)blockIdx.x * kRows, m0 = (int)blockIdx.y * kTok, l = (int)blockIdx.z;
  const int8_t* a = p.a + ((long long)l * p.N + n0) * p.K;
  const int8_t* b = p.b + ((long long)l * p.M + m0) * p.K;

  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;

  const bool a_lo = n0 + g < p.N, a_hi = n0 + g + 8 < p.N;
  for (int k0 = warp * kChunk; k0 < p.K; k0 += kWarps * kChunk) {
    const int k = k0 + 16 * t;
    const uint4 wa = load16(a + (long long)g * p.K, k, p.K, a_lo);
    const uint4 wb = load16(a + (long long)(g + 8) * p.K, k, p.K, a_hi);
    uint4 x[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) x[i] = load16(b + (long long)(8 * i + g) * p.K, k, p.K, m0 + 8 * i + g < p.M);
    const uint32_t la[4] = {wa.x, wa.y, wa.z, wa.w}, lb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t f[4];
      dev::i8x4_to_f16(la[j], f[0], f[2]);
      dev::i8x4_to_f16(lb[j], f[1], f[3]);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        uint32_t b0, b1;
        dev::i8x4_to_f16(j == 0 ? x[i].x : j == 1 ? x[i].y : j == 2 ? x[i].z : x[i].w, b0, b1);
        mma_f16(acc[i], f, b0, b1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    s_part[warp][g][8 * i + 2 * t] = acc[i][0];
    s_part[warp][g][8 * i + 2 * t + 1] = acc[i][1];
    s_part[warp][g + 8][8 * i + 2 * t] = acc[i][2];
    s_part[warp][g + 8][8 * i + 2 * t + 1] = acc[i][3];
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < kRows * kTok; i += 32 * kWarps) {
    const int r = i % kRows, m = m0 + i / kRows, n = n0 + r;
    if (m >= p.M || n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_part[w][r][i / kRows];
    store_i8_result(p, l, m, n, v);
  }
}

template <int kTok>
cudaError_t launch_stream(const I8Params& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + kRows - 1) / kRows), (unsigned)((p.M + kTok - 1) / kTok), (unsigned)p.L);
  return launch_chained(i8_stream_kernel<kTok>, grid, dim3(32 * kWarps), 0, 1, stream, p);
}

}  // namespace

cudaError_t launch_i8_stream(const I8Params& p, const I8Plan& plan, cudaStream_t stream) {
  switch (plan.tokens) {
    case 8: return launch_stream<8>(p, stream);
    case 16: return launch_stream<16>(p, stream);
    default: return launch_stream<32>(p, stream);
  }
}

}  // namespace splitk
