// splitk_gemm_i8(): argument checks and the choice of kernel for the product
// of 8-bit codes.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "splitk.h"
#include "splitk_i8.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

// What a launch of `tiles` tiles costs, in microseconds: rounds of as many
// clusters as the device holds at once, each a CTA's K tiles and a fixed share
// (set-up, first loads, epilogue; more when ranks exchange sums).  Measured on
// GB300: a K tile of 256 tokens 0.53 (the MMAs), of up to 128 0.36 (shared
// memory, conversion, and memory with all SMs at it); fixed 9.5 and 4.6, with a
// split 2 more.
double tile_us(long long tiles, int tokens, int k_tiles, int split, const int (&clusters)[4]) {
  const int fit = clusters[split - 1];
  if (tiles == 0) return 0.0;
  if (fit <= 0 || split > k_tiles) return 1e30;
  const double rounds = (double)((tiles + fit - 1) / fit);
  const double each = (tokens == 256 ? 0.53 : 0.36) * ((k_tiles + split - 1) / split);
  return rounds * (each + (tokens == 256 ? 9.5 : 4.6) + (split > 1 ? 2.0 : 0.0));
}

// The tile plan with the least estimated time: all tiles on `split` pairs, or
// as many full rounds of whole tiles as there are and the rest split.
double plan_tiles(int M, int N, int K, int L, const DeviceSize& dev, I8Plan* out) {
  const int k_tiles = (K + 127) / 128;
  double best = 1e30;
  for (int tokens : {32, 64, 128, 256}) {
    if (tokens < 256 && tokens < M && tokens < 128) continue;       // the smallest that holds M, or 128 or 256
    if (tokens > 32 && tokens / 2 >= M) continue;
    const long long tiles = (long long)((M + tokens - 1) / tokens) * ((N + 255) / 256) * L;
    const long long fit = dev.i8_clusters[0];
    const long long rounds = fit > 0 ? tiles / fit : 0;
    for (int split : {1, 2, 3, 4}) {
      const double all = tile_us(tiles, tokens, k_tiles, split, dev.i8_clusters);
      if (all < best) best = all, *out = I8Plan{tokens, 0, split};
      const double rest = tile_us(rounds * fit, tokens, k_tiles, 1, dev.i8_clusters) +
                          tile_us(tiles - rounds * fit, tokens, k_tiles, split, dev.i8_clusters);
      if (split > 1 && rounds > 0 && rest < best) best = rest, *out = I8Plan{tokens, rounds * fit, split};
    }
  }
  return best;
}

// Whether the weights stream through registers, 16 rows and up to 32 tokens a
// CTA: up to 8 tokens always (no tile is filled that far), more where that is
// estimated faster.  Its measured rate is 4.7 TB/s for two token fragments a
// warp, 2.6 for four (each weight is converted once, each token fragment for every
// 16 weight rows).  With four, two CTAs an SM take 1 us and 1.25 for each 1024 of K
// (streamed and in tiles: 17 x 2048 x 16384 23.1 us and 15.5, 17 x 18432 x 256 9.2
// and 5.2, 64 x 2048 x 1024 3.9 and 6.9, 256 x 500 x 4096 7.8 and 9.5; of 150 sizes from
// 33 x 64 x 64 to 1000 x 4096 x 4096 one is chosen wrongly by more than 3 %: 64 x 4096 x
// 1024 6.4 and 6.2).
bool streams(int M, int N, int K, int L, double tile_time, int num_sms) {
  if (M <= 8) return true;
  const double codes = (double)N * K * L;
  if (M <= 16) return 2.5 + codes / 4.7e6 < tile_time;
  const long long blocks = (M + 31) / 32;
  if (blocks > 65535) return false;                    // CTAs of a launch's y dimension
  const long long rounds = (blocks * ((N + 15) / 16) * L + 2 * num_sms - 1) / (2 * num_sms);
  return std::max(2.5 + blocks * codes / 2.6e6, 2.0 + rounds * (1.0 + 1.25 * ((K + 1023) / 1024))) < tile_time;
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
  // (M rounded up to whole tiles stays an int)
  if (M < 1 || N < 1 || K < 1 || L < 1 || K % 16 != 0 || L > 65535 || N > 65535 * 128 || K > (1 << 30) || M > (1 << 30)) {
    return SPLITK_ERR_INVALID_SHAPE;
  }
  // tiles of 128 tokens by 256 weight rows, eight CTAs each at most
  if (((long long)M + 127) / 128 * ((N + 255) / 256) * L > (1ll << 27)) return SPLITK_ERR_INVALID_SHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(bias, 2) ||
      !aligned(c, c_type == SPLITK_DTYPE_F32 ? 4u : 2u)) {
    return SPLITK_ERR_MISALIGNED;
  }
  DeviceSize dev;
  int rc = require_i8(&dev);
  if (rc != SPLITK_OK) return rc;
  const I8Params p{static_cast<const int8_t*>(a_q), static_cast<const int8_t*>(b_q), a_scale, b_scale,
                   static_cast<const uint16_t*>(bias), c, c_type == SPLITK_DTYPE_F32, M, N, K, L};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  I8Plan plan{};
  const double tile_time = plan_tiles(M, N, K, L, dev, &plan);
  // (an injected failure is one of tiles; a streamed product has no wait to fail)
  const I8Waits waits{wait_limit_ns(), injected()};
  if ((M <= 8 || waits.inject == 0) && streams(M, N, K, L, tile_time, dev.num_sms)) {
    return launched(launch_i8_stream(p, dev.num_sms, s));
  }
  if (plan.tokens == 0) return SPLITK_ERR_NO_FIT;      // no CTA pair of it fits the device
  return launched(launch_i8_tile(p, plan, waits, s));
}

}  // extern "C"
