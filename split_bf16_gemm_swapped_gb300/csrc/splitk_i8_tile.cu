// The product of 8-bit codes for more tokens than registers serve: tcgen05.
//
// A CTA owns 128 weight rows (the MMA's M side) and kTok tokens (its N side).
// TMA brings raw code tiles, 128 codes of K wide, into a ring; conversion
// warps read them from there and leave f16 where the tensor core reads it:
// weights in tensor memory (thread = weight row = TMEM lane), tokens in shared
// memory (K-major, 128-byte swizzle).  One thread issues the MMAs, eight of
// K = 16 a tile, into an f32 accumulator in tensor memory.  Raw tiles are half
// the bytes of f16 ones, so the ring holds twice the K, and the weights' f16
// copies cost no shared-memory bandwidth.
//
// `split` CTAs of a cluster may share one output tile, each taking a
// contiguous run of K tiles; each leaves its f32 sums in its own shared
// memory and then adds one slice of the tokens over the ranks in order.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"
#include "splitk_i8.cuh"
#include "splitk_internal.h"
#include "splitk_kernel_common.cuh"

namespace splitk {

namespace {

constexpr int kBufs = 2;                        // f16 copies of a K tile in flight
constexpr uint32_t kRawA = kMmaM * kCtaK;       // 16 KiB: 128 rows of 128 codes
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t kATmemCols = 64;             // 128 f16 of a lane

__host__ __device__ constexpr int conv_b_warps(int tok) { return tok == 256 ? 8 : 4; }
__host__ __device__ constexpr int tile_threads(int tok) { return 32 * (8 + conv_b_warps(tok)); }
__host__ __device__ constexpr uint32_t raw_b(int tok) { return (uint32_t)tok * kCtaK; }
__host__ __device__ constexpr uint32_t f16_b(int tok) { return (uint32_t)tok * kCtaK * 2u; }
__host__ __device__ constexpr uint32_t acc_cols(int tok) { return tok < 32 ? 32u : (uint32_t)tok; }
__host__ __device__ constexpr uint32_t a_col0(int tok) { return (acc_cols(tok) + 63u) & ~63u; }
__host__ __device__ constexpr uint32_t tile_tmem_cols(int tok) { return pow2_at_least(a_col0(tok) + kBufs * kATmemCols); }
size_t tile_smem(int tok, int stages) {
  return (size_t)kAlignSlack + (size_t)stages * (kRawA + raw_b(tok)) + (size_t)kBufs * f16_b(tok) + kBarBytes;
}

// kind::f16 with f16 operands, both K-major, f32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

struct TileParams {
  I8Params g;
  int split;
  int stages;
  unsigned long long wait_limit_ns;
};

// One arrival of a warp whose lanes have all done their part.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31u) == 0) dev::mbar_arrive(bar);
}

template <int kTok>
__global__ void __launch_bounds__(tile_threads(kTok), 1)
    i8_tile_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                   const TileParams p) {
  constexpr int kConvB = 32 * conv_b_warps(kTok);     // threads converting tokens
  constexpr uint32_t kIdesc = idesc_f16_f32(kMmaM, kTok);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t base = (raw + (kAlignSlack - 1)) & ~(kAlignSlack - 1);
  const int stages = p.stages;
  const uint32_t s_a = base;
  const uint32_t s_b = s_a + (uint32_t)stages * kRawA;
  const uint32_t s_f = s_b + (uint32_t)stages * raw_b(kTok);
  const uint32_t s_bar = s_f + kBufs * f16_b(kTok);
  const uint32_t bar_full = s_bar;                    // [kMaxStages] the raw tile landed
  const uint32_t bar_free = s_bar + 8u * kMaxStages;  // [kMaxStages] every conversion warp has read it
  const uint32_t bar_ready = s_bar + 16u * kMaxStages;          // [kBufs] f16 copies written
  const uint32_t bar_used = bar_ready + 8u * kBufs;             // [kBufs] the MMAs have read them
  const uint32_t bar_acc = bar_used + 8u * kBufs;               // the accumulator is complete
  const uint32_t slot_tmem = bar_acc + 8u, slot_abort = bar_acc + 12u;

  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
  const int split = p.split;
  const int rank = split > 1 ? (int)dev::cluster_ctarank() : 0;
  const int m0 = ((int)blockIdx.x / split) * kTok, n0 = (int)blockIdx.y * kMmaM, l = (int)blockIdx.z;
  const int total = (p.g.K + kCtaK - 1) / kCtaK;
  const int each = total / split, extra = total % split;
  const int k_tiles = each + (rank < extra ? 1 : 0);
  const int kt0 = rank * each + (rank < extra ? rank : extra);
  const Waiter waiter{slot_abort, p.wait_limit_ns};

  if (warp == 3 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      dev::mbar_init(bar_full + 8u * s, 1u);
      dev::mbar_init(bar_free + 8u * s, 4u + conv_b_warps(kTok));
    }
    for (int i = 0; i < kBufs; ++i) {
      dev::mbar_init(bar_ready + 8u * i, 4u + conv_b_warps(kTok));
      dev::mbar_init(bar_used + 8u * i, 1u);
    }
    dev::mbar_init(bar_acc, 1u);
    dev::st_shared_u32(slot_abort, 0u);
    dev::fence_barrier_init();
  } else if (warp == 2) {
    dev::tmem_alloc(slot_tmem, tile_tmem_cols(kTok));
    dev::tmem_relinquish();
    dev::tc_fence_before();
  } else if (warp == 0 && lane == 0) {
    dev::tensormap_prefetch(&a_map);
    dev::tensormap_prefetch(&b_map);
  }
  __syncthreads();
  dev::tc_fence_after();
  // The next kernel may come once this CTA holds its tensor memory.
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const uint32_t tmem = dev::ld_shared_u32(slot_tmem);

  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t stream_once = dev::policy_evict_first(), keep = dev::policy_evict_normal();
      RingPos pos{0, 0u};
      for (int kt = 0; kt < k_tiles; ++kt, pos.advance(1, stages)) {
        const uint32_t s = (uint32_t)pos.index;
        if (kt >= stages && !waiter.wait<false>(bar_free + 8u * s, pos.phase ^ 1u, kRoleWeightTma, kt)) break;
        dev::mbar_arrive_expect_tx(bar_full + 8u * s, kRawA + raw_b(kTok));
        dev::tma_load_3d_hint(s_a + s * kRawA, &a_map, (kt0 + kt) * kCtaK, n0, l, bar_full + 8u * s, stream_once);
        dev::tma_load_3d_hint(s_b + s * raw_b(kTok), &b_map, (kt0 + kt) * kCtaK, m0, l, bar_full + 8u * s, keep);
        ++issued;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint64_t b_desc = dev::smem_desc_sw128(s_f);
      RingPos pos{0, 0u};
      for (int kt = 0; kt < k_tiles; ++kt, pos.advance(1, kBufs)) {
        const uint32_t i = (uint32_t)pos.index;
        if (!waiter.wait<false>(bar_ready + 8u * i, pos.phase, kRoleMma, kt)) break;
        dev::tc_fence_after();
        const uint64_t b_d = dev::smem_desc_advance(b_desc, i * f16_b(kTok));
        const uint32_t a_t = tmem + a_col0(kTok) + i * kATmemCols;
#pragma unroll
        for (int j = 0; j < kCtaK / kMmaK; ++j) {
          dev::mma_bf16_ts(tmem, a_t + 8u * j,
                           dev::smem_desc_advance(b_d, (uint32_t)(j >> 2) * raw_b(kTok) + (uint32_t)(j & 3) * 32u),
                           kIdesc, (kt | j) != 0 ? 1u : 0u);
        }
        dev::mma_commit(bar_used + 8u * i);
      }
      dev::mma_commit(bar_acc);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // weights: thread = row = TMEM lane
    const uint32_t row = threadIdx.x - 128u;
    const uint32_t t_row = tmem + a_col0(kTok) + ((row & ~31u) << 16);
    RingPos in{0, 0u}, out{0, 0u};
    for (int kt = 0; kt < k_tiles; ++kt, in.advance(1, stages), out.advance(1, kBufs)) {
      if (!__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_full + 8u * in.index, in.phase, kRoleEpiDecode, kt))) break;
      const uint32_t src = s_a + (uint32_t)in.index * kRawA + row * kCtaK;
      uint32_t c[8][4];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) dev::ld_shared_v4(src + ((j ^ (row & 7u)) << 4), c[j][0], c[j][1], c[j][2], c[j][3]);
      warp_arrive(bar_free + 8u * in.index);
      if (kt >= kBufs &&
          !__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_used + 8u * out.index, out.phase ^ 1u, kRoleEpiDecode, kt))) break;
      dev::tc_fence_after();
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t f[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) dev::i8x4_to_f16(c[2 * h + (j >> 2)][j & 3], f[2 * j], f[2 * j + 1]);
        dev::tmem_st_x16(t_row + (uint32_t)out.index * kATmemCols + 16u * h, f);
      }
      dev::tmem_wait_st();
      dev::tc_fence_before();
      warp_arrive(bar_ready + 8u * out.index);
    }
  } else if (warp >= 8) {
    // tokens: kConvB / kTok threads a row, chunks of 16 codes
    constexpr int kPer = 8 * kTok / kConvB;           // chunks a thread converts
    const uint32_t t = threadIdx.x - 256u, row = t % kTok, first = (t / kTok) * kPer;
    RingPos in{0, 0u}, out{0, 0u};
    for (int kt = 0; kt < k_tiles; ++kt, in.advance(1, stages), out.advance(1, kBufs)) {
      if (!__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_full + 8u * in.index, in.phase, kRoleEpiDecode, kt))) break;
      const uint32_t src = s_b + (uint32_t)in.index * raw_b(kTok) + row * kCtaK;
      uint32_t c[kPer][4];
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) {
        dev::ld_shared_v4(src + (((first + j) ^ (row & 7u)) << 4), c[j][0], c[j][1], c[j][2], c[j][3]);
      }
      warp_arrive(bar_free + 8u * in.index);
      if (kt >= kBufs &&
          !__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_used + 8u * out.index, out.phase ^ 1u, kRoleEpiDecode, kt))) break;
      const uint32_t dst = s_f + (uint32_t)out.index * f16_b(kTok) + row * 128u;
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) {
        // 16 codes become two 16-byte chunks of one 64-wide half of the tile
        const uint32_t at = dst + ((first + j) >> 2) * raw_b(kTok), chunk = 2u * ((first + j) & 3u);
        uint32_t f[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) dev::i8x4_to_f16(c[j][w], f[2 * w], f[2 * w + 1]);
        dev::st_shared_v4(at + ((chunk ^ (row & 7u)) << 4), f[0], f[1], f[2], f[3]);
        dev::st_shared_v4(at + (((chunk + 1u) ^ (row & 7u)) << 4), f[4], f[5], f[6], f[7]);
      }
      dev::fence_proxy_async_shared();
      warp_arrive(bar_ready + 8u * out.index);
    }
  }

  // ---- epilogue: every thread waits for the accumulator, warps 4..7 read it
  waiter.wait<false>(bar_acc, 0u, kRoleEpiMma, 0);
  __syncwarp();
  dev::tc_fence_after();
  const int live = min(kTok, p.g.M - m0);
  if (warp >= 4 && warp < 8) {
    const int row = (int)threadIdx.x - 128, n = n0 + row;
    const uint32_t t_row = tmem + ((uint32_t)(row & ~31) << 16);
    for (int g = 0; g * 16 < live; ++g) {
      uint32_t v[16];
      __syncwarp();
      dev::tmem_ld_x16(t_row + 16u * g, v);
      dev::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int col = g * 16 + e;
        if (split > 1) {
          dev::st_shared_u32(base + (uint32_t)(col * kMmaM + row) * 4u, v[e]);
        } else if (col < live && n < p.g.N) {
          store_i8_result(p.g, l, m0 + col, n, __uint_as_float(v[e]));
        }
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
    const int c0 = live * rank / split, c1 = live * (rank + 1) / split;
    for (int i = (int)threadIdx.x; i < (c1 - c0) * kMmaM; i += tile_threads(kTok)) {
      const int col = c0 + i / kMmaM, row = i % kMmaM;
      const uint32_t at = base + (uint32_t)(col * kMmaM + row) * 4u;
      float v = 0.0f;
      for (int r = 0; r < split; ++r) v += dev::ld_cluster_f32(dev::mapa(at, (uint32_t)r));
      if (n0 + row < p.g.N) store_i8_result(p.g, l, m0 + col, n0 + row, v);
    }
    __syncwarp();
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
  }

  // ---- teardown.  After a failed wait, copies and MMAs in flight land (for a
  // bounded time) before the CTA gives up its memory.
  if (dev::ld_shared_u32(slot_abort) != 0u) {
    const unsigned long long drain_ns = 10000000ull;   // 10 ms
    if (threadIdx.x == 0) {
      for (int s = 0; s < issued && s < stages; ++s) {
        drain_wait(bar_full + 8u * s, (uint32_t)(((issued - 1 - s) / stages) & 1), drain_ns);
      }
    }
    if (warp == 2) drain_wait(bar_acc, 0u, drain_ns);
  }
  dev::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, tile_tmem_cols(kTok));
  }
}

template <int kTok>
cudaError_t launch_tile(const I8Params& g, int split, int stages, unsigned long long wait_limit_ns, cudaStream_t stream) {
  CUtensorMap a_map, b_map;
  if (!encode_codes(&a_map, g.a, g.K, g.N, g.L, kMmaM) || !encode_codes(&b_map, g.b, g.K, g.M, g.L, kTok)) {
    return cudaErrorInvalidValue;
  }
  const dim3 grid((unsigned)(((g.M + kTok - 1) / kTok) * split), (unsigned)((g.N + kMmaM - 1) / kMmaM), (unsigned)g.L);
  const TileParams p{g, split, stages, wait_limit_ns};
  return launch_chained(i8_tile_kernel<kTok>, grid, dim3(tile_threads(kTok)), tile_smem(kTok, stages), (unsigned)split,
                        stream, a_map, b_map, p);
}

}  // namespace

cudaError_t launch_i8_tile(const I8Params& p, const I8Plan& plan, unsigned long long wait_limit_ns, cudaStream_t stream) {
  switch (plan.tokens) {
    case 32: return launch_tile<32>(p, plan.split, plan.stages, wait_limit_ns, stream);
    case 64: return launch_tile<64>(p, plan.split, plan.stages, wait_limit_ns, stream);
    case 128: return launch_tile<128>(p, plan.split, plan.stages, wait_limit_ns, stream);
    default: return launch_tile<256>(p, plan.split, plan.stages, wait_limit_ns, stream);
  }
}

cudaError_t prepare_i8_tile(int max_dynamic_smem) {
  cudaError_t e;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(i8_tile_kernel<32>, attr, max_dynamic_smem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(i8_tile_kernel<64>, attr, max_dynamic_smem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(i8_tile_kernel<128>, attr, max_dynamic_smem)) != cudaSuccess) return e;
  return cudaFuncSetAttribute(i8_tile_kernel<256>, attr, max_dynamic_smem);
}

cudaError_t read_and_clear_fault_i8(int* out_words) {
  cudaError_t e = cudaMemcpyFromSymbol(out_words, g_fault, sizeof(int) * kFaultWords);
  if (e != cudaSuccess) return e;
  int zeros[kFaultWords] = {0};
  return cudaMemcpyToSymbol(g_fault, zeros, sizeof(zeros));
}

}  // namespace splitk
