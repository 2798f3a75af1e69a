// The product of 8-bit codes for few tokens: the weights stream from memory
// straight into registers.
//
// A CTA owns 16 weight rows (the M side of mma.m16n8k16) and up to 32 tokens
// (its N side), and its warps take the 64-code chunks of K in turn, so
// that a weight row's bytes are read as whole lines.  K is the sum's index, so
// its order within a chunk is free: lane t of each group of four takes the 16
// bytes [16 t, 16 t + 16) of a row, and word j of them is the lane's share of
// the chunk's j-th product for weights and tokens alike.  Neither operand
// passes through shared memory, and a 16-byte load needs no shuffle.
//
// Memory bounds it: 18432 x 7168 codes take 23.2 us for one token, 5.7 TB/s.  The
// loads in flight are what brings it there, so none hangs on a branch.
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
constexpr int kPrefetch = 1024;      // codes of a row
constexpr int kChunk = 64;           // codes of K a warp takes at a time
constexpr int kAhead = 2;            // chunks whose loads a warp has in flight at once

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// kTok: token columns of a CTA (8, 16 or 32).  kWarps: its warps, 8 or 16.
template <int kTok, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kWarps / 8) i8_stream_kernel(const I8Params p) {
  constexpr int kTiles = kTok / 8;
  __shared__ float s_part[kWarps][kRows][kTok + 1];
  dev::griddep_launch_dependents();
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = (int)blockIdx.x * kRows, m0 = (int)blockIdx.y * kTok, l = (int)blockIdx.z;
  // While the work ahead in the stream completes, the rows' first codes come to
  // L2 (which is where a kernel's writes would change them: nothing is read early).
  // (1 x 7168 x 2048: 5.1 us without, 4.6; whole rows of 7168: slower again, they
  // displace what other CTAs are loading.)
  if ((int)threadIdx.x < kRows && n0 + (int)threadIdx.x < p.N && blockIdx.y == 0) {
    dev::prefetch_l2(p.a + ((long long)l * p.N + n0 + (int)threadIdx.x) * p.K, (uint32_t)min(p.K, kPrefetch));
  }
  dev::griddep_wait();
  // Rows and tokens past the end read the last one instead (their sums are not
  // stored), and the last chunk's lanes past K read in front of it and count
  // as zeros: no load hangs on a branch.
  const int8_t* a[2];
  const int8_t* b[kTiles];
#pragma unroll
  for (int r = 0; r < 2; ++r) a[r] = p.a + ((long long)l * p.N + min(n0 + 8 * r + g, p.N - 1)) * p.K;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) b[i] = p.b + ((long long)l * p.M + min(m0 + 8 * i + g, p.M - 1)) * p.K;

  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;

  for (int k0 = warp * kChunk; k0 < p.K; k0 += kAhead * kWarps * kChunk) {
    uint4 w[kAhead][2], x[kAhead][kTiles];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = min(k0 + u * kWarps * kChunk + 16 * t, p.K - 16);
#pragma unroll
      for (int r = 0; r < 2; ++r) w[u][r] = *reinterpret_cast<const uint4*>(a[r] + at);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) x[u][i] = *reinterpret_cast<const uint4*>(b[i] + at);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k0 + u * kWarps * kChunk + 16 * t >= p.K) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) x[u][i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t q[4];
        dev::i8x4_to_f16(word(w[u][0], j), q[0], q[2]);
        dev::i8x4_to_f16(word(w[u][1], j), q[1], q[3]);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          uint32_t f0, f1;
          dev::i8x4_to_f16(word(x[u][i], j), f0, f1);
          mma_f16(acc[i], q, f0, f1);
        }
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
  const int live = min(kTok, p.M - m0), r = (int)threadIdx.x % kRows, n = n0 + r;
  const I8Channel channel(p, l, n);
  const float* scales = p.b_scale + (long long)l * p.M + m0;
  for (int c = (int)threadIdx.x / kRows; c < live; c += 32 * kWarps / kRows) {
    const float scale = scales[c];
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_part[w][r][c];
    if (n < p.N) store_i8_result(p, l, m0 + c, n, v, scale, channel);
  }
}

template <int kTok>
cudaError_t launch_stream(const I8Params& p, int num_sms, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + kRows - 1) / kRows), (unsigned)((p.M + kTok - 1) / kTok), (unsigned)p.L);
  // Up to two CTAs an SM get twice the warps, for more loads in flight, where K
  // gives each warp more than a chunk or two (one token, 4096 x 7168: 11.0 us with
  // eight, 8.5 with sixteen; 18432 x 7168: 23.4 and 27.9; 2048 x 1024: 2.3 and 2.7).
  // 32 tokens would not fit their registers.
  if constexpr (kTok < 32) {
    if ((long long)grid.x * grid.y * grid.z <= 2ll * num_sms && p.K > 2048) {
      return launch_chained(i8_stream_kernel<kTok, 16>, grid, dim3(32 * 16), 0, 1, stream, p);
    }
  }
  return launch_chained(i8_stream_kernel<kTok, 8>, grid, dim3(32 * 8), 0, 1, stream, p);
}

}  // namespace

cudaError_t launch_i8_stream(const I8Params& p, int num_sms, cudaStream_t stream) {
  if (p.M <= 8) return launch_stream<8>(p, num_sms, stream);
  if (p.M <= 16) return launch_stream<16>(p, num_sms, stream);
  return launch_stream<32>(p, num_sms, stream);
}

}  // namespace splitk
