// The product of 8-bit codes for more tokens than registers serve: tcgen05 on
// pairs of SMs.
//
// A pair of CTAs owns 256 weight rows (the M side of a cta_group::2 MMA, 128 in
// each CTA's tensor memory) and kTok tokens (its N side, half of them in each
// CTA's shared memory).  TMA brings raw code tiles, 128 codes of K wide, into a
// ring; conversion warps read them from there and leave f16 where the tensor
// core reads it: weights in tensor memory (thread = weight row = TMEM lane),
// tokens in shared memory (K-major, 128-byte swizzle).  The leader CTA issues
// the MMAs, eight of K = 16 a tile, for both.
//
// What bounds it is shared-memory bandwidth, 128 bytes a clock and SM: a K tile
// costs the arrival and the reading of the raw codes, and the writing and the
// MMA's reading of the tokens' f16 (the weights' f16 never pass through it).
// A pair halves the token side for each SM.  With one CTA a tile, 128 tokens
// took ~1,050 clocks a K tile (1,024 by that count; 512 the MMAs alone).  Pairs
// take ~690 for 128 tokens, and ~1,020 for 256, where the MMAs (1,024) bound it:
// 1000 x 7168 x 16384 in 128 us, 94 % of the measured bf16 rate (one call after another
// runs into the power cap: 139).  Up to 64 tokens the weights' arrival bounds it: 64 x
// 18432 x 7168 in 25.3 us, 80 % of the copy rate (5 us of that before the first MMA and
// after the last).
//
// `split` pairs of a cluster may share one output tile, each taking a
// contiguous run of K tiles; each CTA leaves its f32 sums in its own shared
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

constexpr uint32_t kRawA = kMmaM * kCtaK;       // 16 KiB: 128 rows of 128 codes
constexpr uint32_t kBarBytes = 256;
constexpr uint32_t kATmemCols = 64;             // 128 f16 of a lane
// Two groups of warps convert, each every other K tile: a group's tile is a
// chain of latencies (wait, shared loads, conversion, tensor-memory stores,
// fence) that one group alone could not hide.  A ring slot belongs to one
// group (slot counts are even), so that a group meets every phase of its
// barriers.
constexpr int kGroups = 2;
constexpr int kGroupWarps = 4;
constexpr int kConvA0 = 4, kConvB0 = kConvA0 + kGroups * kGroupWarps;     // first warps of the conversion groups
constexpr int kTileThreads = 32 * (kConvB0 + kGroups * kGroupWarps);

// Tokens whose codes one CTA of a pair converts.
__host__ __device__ constexpr int half_of(int tok) { return tok / 2; }
// f16 copies of a K tile in flight
__host__ __device__ constexpr int bufs(int tok) { return tok <= 128 ? 4 : 2; }
// MMA issuers, each with an accumulator of its own: an MMA takes ~90 clocks to
// issue beside busy conversion warps, so that one thread would bound tiles of
// up to 128 tokens (64 clocks of tensor core an MMA).
__host__ __device__ constexpr int issuers(int tok) { return tok <= 128 ? 2 : 1; }
__host__ __device__ constexpr uint32_t raw_b(int tok) { return (uint32_t)half_of(tok) * kCtaK; }
__host__ __device__ constexpr uint32_t f16_b(int tok) { return (uint32_t)half_of(tok) * kCtaK * 2u; }
__host__ __device__ constexpr uint32_t acc_cols(int tok) { return tok < 32 ? 32u : (uint32_t)tok; }
__host__ __device__ constexpr uint32_t a_col0(int tok) { return ((uint32_t)issuers(tok) * acc_cols(tok) + 63u) & ~63u; }
// All of the tensor memory: one CTA an SM whatever the tile.
constexpr uint32_t kTileTmemCols = 512;
// Raw tiles in flight: what shared memory holds beside the f16 copies (an even
// number, one SM a CTA).
__host__ __device__ constexpr int ring_stages(int tok) { return tok <= 128 ? 6 : 4; }
size_t tile_smem(int tok) {
  return (size_t)kAlignSlack + (size_t)ring_stages(tok) * (kRawA + raw_b(tok)) + (size_t)bufs(tok) * f16_b(tok) + kBarBytes +
         (size_t)tok * sizeof(float);
}

// kind::f16 with f16 operands, both K-major, f32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T over the pair of CTAs, and the arrival of
// what was issued so far on both CTAs' mbarriers, of the one lane of a converged
// warp whose `leader` is 1.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar, uint32_t cta_mask, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      ".reg .b16 m;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "cvt.u16.u32 m, %1;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          bar),
      "r"(cta_mask), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

struct TileParams {
  I8Params g;
  int split;
  long long tile0;          // the launch's first tile
  I8Waits waits;
  bool quads;               // C may be stored four channels at a time
};

// One arrival of a warp whose lanes have all done their part.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31u) == 0) dev::mbar_arrive(bar);
}

// A raw slot whose codes the warp has loaded is free for the next tile's copy.
// The copy is of the async proxy, and an arrival alone does not hold it back
// until loads that are still under way have read the slot: each lane's fence does.
__device__ __forceinline__ void warp_free(uint32_t bar) {
  dev::fence_proxy_async_shared();
  warp_arrive(bar);
}

// An arrival on a barrier of the pair's leader, which issues the MMAs that read what
// the warp has written to this CTA's memories.  For tensor memory the arrival is
// enough: the tcgen05 fences on either side order it.  Shared memory (fenced to
// the async proxy by each lane) is released at cluster scope, which the leader's
// wait acquires at; by a fence of shared memory alone, since an arrival's own
// release waits ~1,250 clocks for every outstanding memory operation (1000 x 7168 x
// 16384: 268 us then, or 150 with threads of their own to release it).
__device__ __forceinline__ void warp_arrive_pair(uint32_t cluster_bar, bool shared) {
  __syncwarp();
  if ((threadIdx.x & 31u) == 0) {
    if (shared) dev::fence_release_shared_cluster();
    dev::mbar_arrive_remote_relaxed(cluster_bar);
  }
}

template <int kTok>
__global__ void __launch_bounds__(kTileThreads, 1)
    i8_tile_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                   const TileParams p) {
  constexpr int kBufs = bufs(kTok);
  constexpr int kIssuers = issuers(kTok);
  constexpr uint32_t kIdesc = idesc_f16_f32(2 * kMmaM, kTok);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t base = (raw + (kAlignSlack - 1)) & ~(kAlignSlack - 1);
  constexpr int stages = ring_stages(kTok);
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
  const uint32_t s_scale = s_bar + kBarBytes;                   // [kTok] the tokens' scales

  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
  const int split = p.split;
  // cluster rank 2 r + half: CTA `half` of the pair that takes K slice r
  const int cta = (int)dev::cluster_ctarank(), half = cta & 1, rank = cta >> 1;
  const long long tile = p.tile0 + (int)blockIdx.x / (2 * split);
  const int m_tiles = (p.g.M + kTok - 1) / kTok, n_tiles = (p.g.N + 2 * kMmaM - 1) / (2 * kMmaM);
  const int m0 = (int)(tile % m_tiles) * kTok, l = (int)(tile / m_tiles / n_tiles);
  const int n0 = (2 * (int)(tile / m_tiles % n_tiles) + half) * kMmaM;
  const int total = (p.g.K + kCtaK - 1) / kCtaK;
  const int each = total / split, extra = total % split;
  const int k_tiles = each + (rank < extra ? 1 : 0);
  const int kt0 = rank * each + (rank < extra ? rank : extra);
  const Waiter waiter{slot_abort, p.waits.limit_ns};
  const bool report = half == 0 || (p.waits.inject & kInjectSkipPublish) == 0;

  if (warp == 3 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      dev::mbar_init(bar_full + 8u * s, 1u);
      dev::mbar_init(bar_free + 8u * s, 2u * kGroupWarps);
    }
    for (int i = 0; i < kBufs; ++i) {
      dev::mbar_init(bar_ready + 8u * i, 4u * kGroupWarps);   // both CTAs' (the leader's is the one used)
      dev::mbar_init(bar_used + 8u * i, 1u);
    }
    dev::mbar_init(bar_acc, kIssuers);
    dev::st_shared_u32(slot_abort, 0u);
    dev::fence_barrier_init();
  } else if (warp == 2) {
    tmem_alloc_pair(slot_tmem, kTileTmemCols);
    dev::tc_fence_before();
  } else if (warp == 0 && lane == 0) {
    dev::tensormap_prefetch(&a_map);
    dev::tensormap_prefetch(&b_map);
  }
  __syncwarp();
  dev::cluster_arrive_release();
  dev::cluster_wait_acquire();
  dev::tc_fence_after();
  // The next kernel may come once this CTA holds its tensor memory.
  dev::griddep_launch_dependents();
  // While the work ahead in the stream completes, the ring's first weight tiles
  // come to L2 (which is where a kernel's writes would change them: nothing is
  // read early).
  if (warp == 0 && lane < min(stages, k_tiles)) dev::tma_prefetch_3d(&a_map, (kt0 + lane) * kCtaK, n0, l);
  dev::griddep_wait();
  const uint32_t tmem = dev::ld_shared_u32(slot_tmem);

  const uint32_t ready_of_leader = dev::mapa(bar_ready, (uint32_t)(cta & ~1));

  const int live = min(kTok, p.g.M - m0);
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
        dev::tma_load_3d_hint(s_b + s * raw_b(kTok), &b_map, (kt0 + kt) * kCtaK, m0 + half * half_of(kTok), l, bar_full + 8u * s, keep);
        ++issued;
      }
    }
    __syncwarp();
  } else if (warp >= 1 && warp <= kIssuers) {
    // The whole warp of the leader CTA walks the tiles and one lane's predicate
    // lets the instructions through.
    if (half == 0) {
      const int first = warp - 1;
      const uint32_t leader = lane == 0 ? 1u : 0u;
      const uint32_t both = 3u << (2 * rank);
      const uint64_t b_desc = dev::smem_desc_sw128(s_f);
      const uint32_t base_col = __shfl_sync(0xFFFFFFFFu, tmem, 0), acc = base_col + (uint32_t)first * acc_cols(kTok);
      RingPos pos = RingPos::at(first, kBufs);
      for (int kt = first; kt < k_tiles; kt += kIssuers, pos.advance(kIssuers, kBufs)) {
        const uint32_t i = (uint32_t)pos.index;
        if (!__all_sync(0xFFFFFFFFu, waiter.wait<true>(bar_ready + 8u * i, pos.phase, kRoleMma, kt))) break;
        dev::tc_fence_after();
        const uint64_t b_d = dev::smem_desc_advance(b_desc, i * f16_b(kTok));
        const uint32_t a_t = base_col + a_col0(kTok) + i * kATmemCols;
#pragma unroll
        for (int j = 0; j < kCtaK / kMmaK; ++j) {
          mma_pair(acc, a_t + 8u * j,
                   dev::smem_desc_advance(b_d, (uint32_t)(j >> 2) * raw_b(kTok) + (uint32_t)(j & 3) * 32u), kIdesc,
                   (kt >= kIssuers || j != 0) ? 1u : 0u, leader);
        }
        commit_pair(bar_used + 8u * i, both, leader);
      }
      commit_pair(bar_acc, both, leader);
    }
    __syncwarp();
  } else if (warp == 3) {
    for (int c = lane; c < live; c += 32) {
      dev::st_shared_f32(s_scale + 4u * (uint32_t)c, p.g.b_scale[(long long)l * p.g.M + m0 + c]);
    }
  } else if (warp >= kConvA0 && warp < kConvB0) {
    // weights: thread = row = TMEM lane
    const int group = (warp - kConvA0) / kGroupWarps;
    const uint32_t row = (threadIdx.x - 32u * kConvA0) & (kMmaM - 1);
    const uint32_t t_row = tmem + a_col0(kTok) + ((row & ~31u) << 16);
    RingPos in = RingPos::at(group, stages), out = RingPos::at(group, kBufs);
    for (int kt = group; kt < k_tiles; kt += kGroups, in.advance(kGroups, stages), out.advance(kGroups, kBufs)) {
      if (!__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_full + 8u * in.index, in.phase, kRoleEpiDecode, kt))) break;
      const uint32_t src = s_a + (uint32_t)in.index * kRawA + row * kCtaK;
      uint32_t c[8][4];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) {
        dev::ld_shared_v4(src + ((j ^ (row & 7u)) << 4), c[j][0], c[j][1], c[j][2], c[j][3]);
      }
      warp_free(bar_free + 8u * in.index);
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
      if (report) warp_arrive_pair(ready_of_leader + 8u * out.index, false);
    }
  } else if (warp >= kConvB0) {
    // tokens: 128 / half threads a row, each kPer of its 16-code chunks
    constexpr int kRowsB = half_of(kTok), kPer = 8 * kRowsB / 128;
    const int group = (warp - kConvB0) / kGroupWarps;
    const uint32_t t = (threadIdx.x - 32u * kConvB0) & 127u;
    const uint32_t row = t % kRowsB, first = (t / kRowsB) * kPer;
    RingPos in = RingPos::at(group, stages), out = RingPos::at(group, kBufs);
    for (int kt = group; kt < k_tiles; kt += kGroups, in.advance(kGroups, stages), out.advance(kGroups, kBufs)) {
      if (!__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_full + 8u * in.index, in.phase, kRoleEpiDecode, kt))) break;
      const uint32_t src = s_b + (uint32_t)in.index * raw_b(kTok) + row * kCtaK;
      uint32_t c[kPer][4];
#pragma unroll
      for (uint32_t j = 0; j < kPer; ++j) {
        dev::ld_shared_v4(src + (((first + j) ^ (row & 7u)) << 4), c[j][0], c[j][1], c[j][2], c[j][3]);
      }
      warp_free(bar_free + 8u * in.index);
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
      if (report) warp_arrive_pair(ready_of_leader + 8u * out.index, true);
    }
  }

  // ---- epilogue: all sixteen conversion warps read the accumulator, four a
  // TMEM lane quadrant taking 16 tokens in turn
  const int row = (warp & 3) * 32 + lane, n = n0 + row;
  const I8Channel channel(p.g, l, n);
  waiter.wait<false>(bar_acc, 0u, kRoleEpiMma, 0);
  __syncthreads();                                     // and the scales of warp 3
  dev::tc_fence_after();
  if (warp >= kConvA0) {
    const uint32_t t_row = tmem + ((uint32_t)(row & ~31) << 16);
    constexpr int kStep = (kConvB0 - kConvA0) / 2;      // warps a quadrant
    for (int g = (warp - kConvA0) / 4; g * 16 < live; g += kStep) {
      uint32_t v[16];
      __syncwarp();
      load_acc16(t_row + 16u * g, acc_cols(kTok), kIssuers > 1 && k_tiles > 1, v);
      if (split > 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) dev::st_shared_u32(base + (uint32_t)((g * 16 + e) * kMmaM + row) * 4u, v[e]);
      } else {
        uint32_t sc[16];
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          dev::ld_shared_v4(s_scale + 64u * (uint32_t)g + 4u * e, sc[e], sc[e + 1], sc[e + 2], sc[e + 3]);
        }
        const int cols = n < p.g.N ? min(16, live - g * 16) : 0;
        const long long at = ((long long)l * p.g.M + m0 + g * 16) * p.g.N + n;
        if (p.g.c_f32) {
          float* c = static_cast<float*>(p.g.c) + at;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (e < cols) c[(long long)e * p.g.N] = channel.result(__uint_as_float(v[e]), __uint_as_float(sc[e]));
          }
        } else {
          uint16_t* c = static_cast<uint16_t*>(p.g.c) + at;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float r = channel.result(__uint_as_float(v[e]), __uint_as_float(sc[e]));
            if (e < cols) c[(long long)e * p.g.N] = (uint16_t)dev::pack_bf16x2(r, 0.0f);
          }
        }
      }
    }
  }
  if (split > 1) {
    // this rank's slice of the tokens, a column a warp and four weight rows a
    // lane, kAtOnce columns' loads in flight
    constexpr int kAtOnce = 2;
    const int r4 = 4 * lane;
    const I8Channel ch[4] = {I8Channel(p.g, l, n0 + r4), I8Channel(p.g, l, n0 + r4 + 1), I8Channel(p.g, l, n0 + r4 + 2),
                             I8Channel(p.g, l, n0 + r4 + 3)};
    __syncwarp();
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
    const int c0 = live * rank / split, c1 = live * (rank + 1) / split;
    constexpr int kWarpsAll = kTileThreads / 32;
    for (int col = c0 + warp; col < c1; col += kAtOnce * kWarpsAll) {
      float v[kAtOnce][4];
      for (int r = 0; r < split; ++r) {
        float part[kAtOnce][4];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          // (past the slice: the first column again, not used)
          const int c = col + i * kWarpsAll < c1 ? col + i * kWarpsAll : col;
          dev::ld_cluster_f32x4(dev::mapa(base + (uint32_t)(c * kMmaM + r4) * 4u, (uint32_t)(2 * r + half)), part[i]);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] = r == 0 ? part[i][e] : v[i][e] + part[i][e];
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int c = col + i * kWarpsAll;
        if (c >= c1) break;
        const float scale = dev::ld_shared_f32(s_scale + 4u * (uint32_t)c);
        if (p.quads) {                                  // N a multiple of 4, C aligned for it
          if (n0 + r4 >= p.g.N) continue;
          const long long at = ((long long)l * p.g.M + m0 + c) * p.g.N + n0 + r4;
          float o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = ch[e].result(v[i][e], scale);
          if (p.g.c_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(p.g.c) + at) = make_float4(o[0], o[1], o[2], o[3]);
          } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.g.c) + at) =
                make_uint2(dev::pack_bf16x2(o[0], o[1]), dev::pack_bf16x2(o[2], o[3]));
          }
          continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n0 + r4 + e < p.g.N) store_i8_result(p.g, l, m0 + c, n0 + r4 + e, v[i][e], scale, ch[e]);
        }
      }
    }
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
  // No CTA leaves, or frees tensor memory, while another of the cluster may
  // still read its shared memory, arrive on its barriers or run MMAs on it.
  dev::tc_fence_before();
  __syncwarp();
  dev::cluster_arrive_release();
  dev::cluster_wait_acquire();
  if (warp == 2) {
    dev::tc_fence_after();
    tmem_dealloc_pair(tmem, kTileTmemCols);
  }
}

template <int kTok>
cudaError_t launch_tile(const I8Params& g, const I8Plan& plan, const I8Waits& waits, cudaStream_t stream) {
  CUtensorMap a_map, b_map;
  if (!encode_codes(&a_map, g.a, g.K, g.N, g.L, kMmaM) || !encode_codes(&b_map, g.b, g.K, g.M, g.L, half_of(kTok))) {
    return cudaErrorInvalidValue;
  }
  const long long tiles =
      (long long)((g.M + kTok - 1) / kTok) * ((g.N + 2 * kMmaM - 1) / (2 * kMmaM)) * g.L;
  const auto launch = [&](long long first, long long count, int split) {
    const uintptr_t quad = g.c_f32 ? 16u : 8u;
    const TileParams p{g, split, first, waits, g.N % 4 == 0 && (uintptr_t)g.c % quad == 0};
    return launch_chained(i8_tile_kernel<kTok>, dim3((unsigned)(count * 2 * split)), dim3(kTileThreads), tile_smem(kTok),
                          (unsigned)(2 * split), stream, a_map, b_map, p);
  };
  if (plan.whole > 0) {
    const cudaError_t e = launch(0, plan.whole, 1);
    if (e != cudaSuccess) return e;
  }
  return plan.whole < tiles ? launch(plan.whole, tiles - plan.whole, plan.split) : cudaSuccess;
}

template <int kTok>
cudaError_t prepare_tile(int max_dynamic_smem) {
  return cudaFuncSetAttribute(i8_tile_kernel<kTok>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_dynamic_smem);
}

}  // namespace

cudaError_t launch_i8_tile(const I8Params& p, const I8Plan& plan, const I8Waits& waits, cudaStream_t stream) {
  switch (plan.tokens) {
    case 32: return launch_tile<32>(p, plan, waits, stream);
    case 64: return launch_tile<64>(p, plan, waits, stream);
    case 128: return launch_tile<128>(p, plan, waits, stream);
    default: return launch_tile<256>(p, plan, waits, stream);
  }
}

cudaError_t prepare_i8_tile(int max_dynamic_smem, int (&clusters)[4]) {
  cudaError_t e;
  if ((e = prepare_tile<32>(max_dynamic_smem)) != cudaSuccess) return e;
  if ((e = prepare_tile<64>(max_dynamic_smem)) != cudaSuccess) return e;
  if ((e = prepare_tile<128>(max_dynamic_smem)) != cudaSuccess) return e;
  if ((e = prepare_tile<256>(max_dynamic_smem)) != cudaSuccess) return e;
  for (int i = 0; i < 4; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * (i + 1));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tile_smem(256);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2u * (i + 1);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters[i], i8_tile_kernel<256>, &cfg)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t read_and_clear_fault_i8(int* out_words) {
  cudaError_t e = cudaMemcpyFromSymbol(out_words, g_fault, sizeof(int) * kFaultWords);
  if (e != cudaSuccess) return e;
  int zeros[kFaultWords] = {0};
  return cudaMemcpyToSymbol(g_fault, zeros, sizeof(zeros));
}

}  // namespace splitk
