// splitk_gemm_mx4(): the matrix product of two operands in microscaled 4-bit codes
// (splitk_mx4.cuh) on the tensor cores' own instruction for them: E2M1 codes and
// E8M0 scales go in as they are, nothing is converted.
//
// A pair of CTAs owns 256 weight rows (the M side of a cta_group::2 MMA, 128 in each
// CTA's tensor memory) and kTok tokens (its N side, half of them in each CTA's
// shared memory).  TMA brings codes, 256 of K wide, from both operands into a ring of
// shared memory (K-major, 128-byte swizzle); a tile's copies of both CTAs report to
// the leader, where one warp issues the tile's four MMAs of K = 64 for both.
//
// The MMA reads scales from tensor memory: for 128 rows and four blocks of K, column g
// of four holds in lane l, of each lane quadrant, the four codes of row 32 g + l.  Four
// scale warps, a quadrant each, load 32s of rows, a sector of each (four K tiles: a
// load costs the L1 cache a look-up a row, however short), exchange them through
// shared memory and store all of them into their quadrants (2048 x 18432 x 7168 110 us with
// a word of one K tile a lane, 94 with sectors).  (Copies by
// tcgen05.cp keep the tensor pipe from MMAs for ~38 clocks each: six a tile of 256
// tokens, 742 clocks with its MMAs instead of 512.)
//
// What bounds it: few tokens, the weights' arrival (1 x 18432 x 7168 14.1 us, 64 tokens
// 14.4: 5.0 TB/s, of which 3 us before the first MMA and after the last); one token and
// short weights, latency (1 x 7168 x 2048 4.75 us); many tokens, the copies' way from L2.
// An MMA's K = 64 at 256 tokens takes a pair 128 clocks (9.6 PFLOP/s at 1.93 GHz; ~72 for
// up to 128 tokens), but each CTA takes 32 KiB of codes a K tile of 512 clocks, 64
// bytes a clock, which its way from L2 just holds: 2048 x 18432 x 7168 takes 89.5 us (6.0
// PFLOP/s), 77 with no output stored, 71 without scales' loads and half the copies, too,
// and 57 by the MMAs' count; 1000 x 7168 x 16384 50.5 us.  (A CTA alone would bring 48 KiB a tile.)
//
// `split` pairs of a cluster may share one output tile, each taking a contiguous run
// of K tiles; each CTA leaves its f32 sums in its own shared memory and then adds
// one slice of the tokens over the ranks in order.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "splitk.h"
#include "splitk_internal.h"
#include "splitk_kernel_common.cuh"
#include "splitk_mx4.cuh"

namespace splitk {

namespace {

// Warps: 0 copies of codes, 1 MMAs, 2 and 3 set-up, then those that bring scales and
// those that store the output.
// (Four more output warps would leave 128 registers a thread, and what is spilled then
// takes the issuing thread twice its time.)
constexpr int kScale0 = 4, kScaleWarps = 4, kOut0 = kScale0 + kScaleWarps, kOutWarps = 4;
constexpr int kMxThreads = 32 * (kOut0 + kOutWarps);
constexpr int kMaxSplit = 4;                         // pairs of a cluster
constexpr unsigned long long kDrainNs = 10000000ull; // 10 ms

__host__ __device__ constexpr uint32_t mx_acc_cols(int tok) { return tok < 32 ? 32u : (uint32_t)tok; }
__host__ __device__ constexpr uint32_t scale_cols(int tok) { return 8u * (1u + groups_b(tok)); }   // of a K tile

// kind::mxf4: E2M1 operands, both K-major, E8M0 scales for each 32, f32 accumulator;
// the scales of a K = 64 step are the lower (id 0) or upper (id 2) half of a word.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27) | (id << 29);
}

// The tensor cores' instructions of the one lane of a converged warp whose `leader` is 1:
// operands that all lanes hold alike stay in uniform registers (with a branch to one
// lane an MMA took it ~100 clocks to issue).

// D[tmem] (+)= A B^T over the pair of CTAs.
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scale,
                                         uint32_t b_scale, uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate), "r"(leader)
      : "memory");
}

// The arrival of what it has issued so far on the same barrier of all CTAs of a mask.
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

// A box into this CTA's shared memory that reports to a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t cluster_bar,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar), "l"(policy)
      : "memory");
}

// A line of global memory to L2.
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); }

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

struct MxParams {
  const uint8_t* a_scale;   // [L][N][K / 32]
  const uint8_t* b_scale;   // [L][M][K / 32]
  const uint16_t* bias;     // bf16 [L][N], or null
  void* c;                  // bf16 or f32 [L][M][N]
  bool c_f32;
  int M, N, K, L;
  int split, stages;
  int tile0, tile_end;      // the launch's tiles
  uint32_t tmem_cols;
  bool sectors;             // the scales' rows are whole sectors of 32 bytes
  unsigned long long limit_ns;
  unsigned inject;
};

// The scale codes of one row and a group of K tiles, 32 bytes.  kSector: they are a
// sector of memory.  Else they lie somewhere in up to three times 16 bytes, and are cut
// out when they are used, as they may still be on their way before.  (Word by word, two
// loads each: 1300 x 6000 x 4448 73 us.)
template <bool kSector>
struct ScaleRow {
  uint32_t x[kSector ? 8 : 12];
  uint32_t shift;           // bytes before the row's first
  int live;                 // bytes that are the row's
  // Codes [at, limit) of the row at `row` of the array [first, end); limit 0: no row.
  __device__ __forceinline__ void load(const uint8_t* row, int at, int limit, const uint8_t* first, const uint8_t* end) {
    live = limit - at;
    if constexpr (kSector) {
      if (live > 0) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                     : "l"(row + at)
                     : "memory");
      }
    } else {
      shift = (uint32_t)(uintptr_t)(row + at) & 15u;
      const uint8_t* low = row + at - shift;
      const int bytes = live > 0 ? (int)shift + min(live, 32) : 0;       // from `low` on, to the last one wanted
#pragma unroll
      for (int i = 0; i < 12; ++i) x[i] = 0u;
      if (low >= first && low + ((bytes + 15) & ~15) <= end) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (16 * c >= bytes) continue;
          const uint4 v = reinterpret_cast<const uint4*>(low)[c];
          x[4 * c] = v.x, x[4 * c + 1] = v.y, x[4 * c + 2] = v.z, x[4 * c + 3] = v.w;
        }
      } else {                                               // an end of the array: byte by byte
        shift = 0u;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (j < live) x[j / 4] |= (uint32_t)row[at + j] << (8 * (j % 4));
        }
      }
    }
  }
  // The codes, 127 past the limit (the row's codes there are zeros, or it is none).
  __device__ __forceinline__ void words(uint32_t (&w)[2 * kGroup]) const {
    constexpr uint32_t kOnes = 0x7F7F7F7Fu;
    if constexpr (kSector) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = live > 0 ? x[i] : kOnes;
    } else {
      uint32_t y[10], z[9];
#pragma unroll
      for (int i = 0; i < 10; ++i) y[i] = (shift & 8u) != 0u ? x[i + 2] : x[i];
#pragma unroll
      for (int i = 0; i < 9; ++i) z[i] = (shift & 4u) != 0u ? y[i + 1] : y[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = __funnelshift_r(z[i], z[i + 1], 8u * (shift & 3u));
        const int n = live - 4 * i;
        const uint32_t kept = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        w[i] = (v & kept) | (kOnes & ~kept);
      }
    }
  }
};

// One output from its sum.
__device__ __forceinline__ void store_mx(const MxParams& p, long long at, float v) {
  if (p.c_f32) {
    static_cast<float*>(p.c)[at] = v;
  } else {
    static_cast<uint16_t*>(p.c)[at] = (uint16_t)dev::pack_bf16x2(v, 0.0f);
  }
}

// A thread's weight row of kCols consecutive tokens, `pitch` bytes apart from `to` on, the
// first `cols` of them.  (Stores without a branch between them: with a choice of type
// and a check for each, a warp took 125 clocks a store, and 256 tokens 17 us.)
template <int kCols, class F>
__device__ __forceinline__ void store_tokens(uint8_t* to, long long pitch, int cols, F one) {
  if (cols >= kCols) {
#pragma unroll
    for (int e = 0; e < kCols; ++e, to += pitch) one(to, e);
  } else {
#pragma unroll
    for (int e = 0; e < kCols; ++e, to += pitch) {
      if (e < cols) one(to, e);
    }
  }
}

// One output tile of a pair: its place and its run of K in stages' shares.
struct MxTile {
  int m0, n0, l, steps, step0;
  template <int kTok>
  __device__ __forceinline__ static MxTile at(const MxParams& p, int tile, int rank, int half) {
    const int m_tiles = (p.M + kTok - 1) / kTok, n_tiles = (p.N + 2 * kMmaM - 1) / (2 * kMmaM);
    constexpr int kStepK = kTileK * kSub;
    const int total = (p.K + kStepK - 1) / kStepK, each = total / p.split, extra = total % p.split;
    MxTile t;
    t.m0 = (tile % m_tiles) * kTok;
    t.n0 = (2 * (tile / m_tiles % n_tiles) + half) * kMmaM;
    t.l = tile / m_tiles / n_tiles;
    t.steps = each + (rank < extra ? 1 : 0);
    t.step0 = rank * each + (rank < extra ? rank : extra);
    return t;
  }
};

// What the scale warps work with.
struct ScaleRing {
  uint32_t exchange;        // two buffers of kGroup tiles in shared memory
  uint32_t tmem;            // the first stage's columns, of the warp's lane quadrant
  uint32_t bar_full_of_leader, bar_done;
  int stages;
  Waiter waiter;
};

// One scale warp: the CTA's K tiles, of one output tile after another, in groups of
// kGroup.  Its rows' loads of the next group are under way while it stores this one's.
// Two buffers let one barrier of the warps a group do.
template <int kTok, bool kSector>
__device__ __forceinline__ void bring_scales(const MxParams& p, const ScaleRing& r, int tile0, int step, int rank, int half,
                                             int warp, int lane) {
  constexpr int kGroups = groups_b(kTok), kLive = (kTok + 31) / 32;        // 128s and 32s of tokens
  constexpr int kOwn = (kLive + kScaleWarps - 1) / kScaleWarps;            // of which a warp loads at most
  constexpr int kStages = kGroup / kSub;              // whole stages a group
  constexpr int kVecs = 2 * kSub * (1 + kGroups);                          // 16 bytes of a lane, of a stage
  const int blocks = p.K / kMxBlock;
  const uint8_t *a_end = p.a_scale + (long long)p.L * p.N * blocks, *b_end = p.b_scale + (long long)p.L * p.M * blocks;
  MxTile t = MxTile::at<kTok>(p, tile0, rank, half);
  int tile = tile0, kt = 0;                             // where the group to load starts
  // (groups start at multiples of their size: a share of K may begin within its first)
  const int skip = t.step0 * kSub % kGroup, k_tiles = skip + t.steps * kSub;
  const int groups = (k_tiles + kGroup - 1) / kGroup * ((p.tile_end - tile0 + step - 1) / step);
  ScaleRow<kSector> a, b[kOwn];
  const auto load = [&] {
    if (tile >= p.tile_end) return;
    const int at = (t.step0 * kSub - skip + kt) * (kTileK / kMxBlock);
    const int n = t.n0 + lane + 32 * warp;
    a.load(p.a_scale + ((long long)t.l * p.N + n) * blocks, at, n < p.N ? blocks : 0, p.a_scale, a_end);
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
      const int o = 32 * (warp + kScaleWarps * q) + lane, m = t.m0 + o;
      b[q].load(p.b_scale + ((long long)t.l * p.M + m) * blocks, at, o < kTok && m < p.M ? blocks : 0, p.b_scale, b_end);
    }
    kt += kGroup;
    if (kt >= k_tiles) {
      kt = 0, tile += step;
      if (tile < p.tile_end) t = MxTile::at<kTok>(p, tile, rank, half);
    }
  };
  load();
  RingPos pos{0, 0u};
  int used = 0, left = k_tiles;                         // stages before; K tiles of the output tile not stored yet
  bool ok = true;                                       // a warp whose wait failed still meets the others' barriers
  uint32_t buffer = r.exchange;
  for (int group = 0; group < groups; ++group) {
    // word w of a K tile: 512 bytes of A's rows, then of B's each 128
    const uint32_t mine = buffer + 16u * lane + 4u * warp;
    uint32_t w[2 * kGroup];
    a.words(w);
#pragma unroll
    for (int j = 0; j < 2 * kGroup; ++j) dev::st_shared_u32(mine + (j / 2) * scales_of(kTok) + (j % 2) * kScaleAtom, w[j]);
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
      if (kLive < kScaleWarps && warp >= kLive) continue;
      b[q].words(w);
#pragma unroll
      for (int j = 0; j < 2 * kGroup; ++j) {
        dev::st_shared_u32(mine + (j / 2) * scales_of(kTok) + (2u + (j % 2) * kGroups + q) * kScaleAtom, w[j]);
      }
    }
    load();
    dev::named_bar_sync(1, 32 * kScaleWarps);
#pragma unroll 1
    for (int i = left == k_tiles ? skip / kSub : 0; ok && i < kStages && i * kSub < left; ++i, ++used) {
      uint32_t v[kVecs][4];
#pragma unroll
      for (int c = 0; c < kVecs; ++c) {
        dev::ld_shared_v4(buffer + 16u * lane + (uint32_t)i * (kSub * scales_of(kTok)) + c * kScaleAtom, v[c][0], v[c][1], v[c][2],
                          v[c][3]);
      }
      if (used >= r.stages) {                           // the stage's MMAs before
        ok = __all_sync(0xFFFFFFFFu, r.waiter.wait<false>(r.bar_done + 8u * pos.index, pos.phase ^ 1u, kRoleEpiDecode, used));
        if (!ok) break;
      }
      dev::tc_fence_after();
      const uint32_t to = r.tmem + (uint32_t)pos.index * (kSub * scale_cols(kTok));
#pragma unroll
      for (int c = 0; c < kVecs; c += 4) {
        uint32_t x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = v[(c + e / 4) % kVecs][e % 4];
        dev::tmem_st_x16(to + 4u * c, x);
      }
      dev::tmem_wait_st();
      dev::tc_fence_before();
      __syncwarp();
      if (lane == 0 && (p.inject & kInjectSkipPublish) == 0) dev::mbar_arrive_remote_relaxed(r.bar_full_of_leader + 8u * pos.index);
      pos.advance(1, r.stages);
    }
    left = left > kGroup ? left - kGroup : k_tiles;
    buffer = r.exchange + (r.exchange + kGroup * scales_of(kTok) - buffer);
  }
}

// A cluster takes tiles gridDim.x / cluster size apart; with split > 1 one alone
// (its sums go where the ring was, below the barriers).
template <int kTok>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map, const MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (dev::smem_u32(smem_raw) + (kAlignSlack - 1)) & ~(kAlignSlack - 1);
  const int stages = p.stages, split = p.split;
  const uint32_t s_a = base;
  const uint32_t s_b = s_a + (uint32_t)stages * kSub * kCodesA;
  const uint32_t s_s = s_b + (uint32_t)stages * kSub * codes_b(kTok);
  const uint32_t s_bar = base + mx_bars_at(kTok, stages, split);
  const uint32_t bar_full = s_bar;                          // [kMxStages] leader: both CTAs' codes and scales are there
  const uint32_t bar_done = bar_full + 8u * kMxStages;      // [kMxStages] the MMAs have read them
  const uint32_t bar_half = bar_done + 8u * kMxStages;      // [kMxStages] those of the first of two K tiles have read it
  const uint32_t bar_acc = bar_half + 8u * kMxStages;       // a tile's accumulator is complete
  const uint32_t bar_read = bar_acc + 8u;                   // leader: both CTAs' output warps have read it
  const uint32_t slot_tmem = bar_read + 8u, slot_abort = slot_tmem + 4u;

  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
  // cluster rank 2 r + half: CTA `half` of the pair that takes K slice r
  const int cta = (int)dev::cluster_ctarank(), half = cta & 1, rank = cta >> 1;
  const int tile0 = p.tile0 + (int)blockIdx.x / (2 * split), step = (int)gridDim.x / (2 * split);
  const Waiter waiter{slot_abort, p.limit_ns};

  if (warp == 3 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      dev::mbar_init(bar_full + 8u * s, 1u + 2u * kScaleWarps);
      dev::mbar_init(bar_done + 8u * s, 1u);
      dev::mbar_init(bar_half + 8u * s, 1u);
    }
    dev::mbar_init(bar_acc, 1u);
    dev::mbar_init(bar_read, 2u * kOutWarps);
    dev::st_shared_u32(slot_abort, 0u);
    dev::fence_barrier_init();
  } else if (warp == 2) {
    tmem_alloc_pair(slot_tmem, p.tmem_cols);
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
  const MxTile tile_first = MxTile::at<kTok>(p, tile0, rank, half);
  // While the work ahead in the stream completes, the ring's first weight tiles and
  // the first of their scales come to L2 (which is where a kernel's writes would change them: nothing is read early).
  if (warp == 0 && lane < min(stages, tile_first.steps) * kSub) {
    dev::tma_prefetch_3d(&a_map, (tile_first.step0 * kSub + lane) * (kTileK / 2), tile_first.n0, tile_first.l);
  }
  if (warp == kScale0) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int n = tile_first.n0 + lane + 32 * g;
      if (n < p.N) {
        prefetch_line(p.a_scale + ((long long)tile_first.l * p.N + n) * (p.K / kMxBlock) +
                      tile_first.step0 * kSub * (kTileK / kMxBlock));
      }
    }
  }
  dev::griddep_wait();
  const uint32_t tmem = dev::ld_shared_u32(slot_tmem);
  const uint32_t leader = (uint32_t)(cta & ~1);

  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t keep = dev::policy_evict_normal(), policy_a = p.M <= kTok ? dev::policy_evict_first() : keep;
      const uint32_t full_of_leader = dev::mapa(bar_full, leader);
      RingPos pos{0, 0u};
      bool ok = true;
      for (int tile = tile0; ok && tile < p.tile_end; tile += step) {
        const MxTile t = MxTile::at<kTok>(p, tile, rank, half);
        for (int i = 0; i < t.steps; ++i, pos.advance(1, stages)) {
          const uint32_t s = (uint32_t)pos.index, bar = full_of_leader + 8u * s;
          const bool again = issued >= stages;
#pragma unroll
          for (int j = 0; j < kSub; ++j) {
            if (again) {
              ok = ok && waiter.wait<false>((j == 0 ? bar_half : bar_done) + 8u * s, pos.phase ^ 1u, kRoleWeightTma, i);
            }
            if (!ok) break;
            if (j == 0) {
              ++issued;
              if (half == 0) dev::mbar_arrive_expect_tx(bar_full + 8u * s, 2u * stage_bytes(kTok));
            }
            const int k = ((t.step0 + i) * kSub + j) * (kTileK / 2);
            tma_load_pair(s_a + (s * kSub + j) * kCodesA, &a_map, k, t.n0, t.l, bar, policy_a);
            tma_load_pair(s_b + (s * kSub + j) * codes_b(kTok), &b_map, k, t.m0 + half * (kTok / 2), t.l, bar, keep);
          }
          if (!ok) break;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // (the whole warp of the leader CTA walks the tiles)
    if (half == 0) {
      RingPos pos{0, 0u};
      const uint32_t both = 3u << (2 * rank), one = lane == 0 ? 1u : 0u;
      const uint64_t a_desc = dev::smem_desc_sw128(s_a), b_desc = dev::smem_desc_sw128(s_b);
      const uint32_t acc = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const auto met = [&](bool done) { return __all_sync(0xFFFFFFFFu, done) != 0; };
      const auto landed = [&](int i) { return met(waiter.wait<true>(bar_full + 8u * pos.index, pos.phase, kRoleMma, i)); };
      uint32_t turn = 0u;
      bool ok = true;
      for (int tile = tile0; ok && tile < p.tile_end; tile += step, ++turn) {
        const MxTile t = MxTile::at<kTok>(p, tile, rank, half);
        ok = landed(0) && (turn == 0u || met(waiter.wait<true>(bar_read, (turn - 1u) & 1u, kRoleMmaAccFree, (int)turn)));
        for (int i = 0; ok && i < t.steps; ++i) {
          dev::tc_fence_after();
          const uint32_t s = (uint32_t)pos.index;
          const uint32_t t_s = acc + mx_acc_cols(kTok) + s * (kSub * scale_cols(kTok));
          const uint64_t a_d = dev::smem_desc_advance(a_desc, s * (kSub * kCodesA));
          const uint64_t b_d = dev::smem_desc_advance(b_desc, s * (kSub * codes_b(kTok)));
          pos.advance(1, stages);
          // (64s of K that there are)
          const int chunks = min(4 * kSub, (p.K - (t.step0 + i) * (kSub * kTileK) + 63) / 64);
#pragma unroll
          for (int j = 0; j < 4 * kSub; ++j) {
            const uint32_t sub = j / 4, t_a = t_s + sub * scale_cols(kTok) + 4u * (j % 4 / 2);
            const uint32_t t_b = t_s + sub * scale_cols(kTok) + 8u + 4u * groups_b(kTok) * (j % 4 / 2);
            if (j < chunks) {
              mma_mxf4(acc, dev::smem_desc_advance(a_d, sub * kCodesA + 32u * (j % 4)),
                       dev::smem_desc_advance(b_d, sub * codes_b(kTok) + 32u * (j % 4)),
                       j % 2 == 0 ? idesc_mxf4(2 * kMmaM, kTok, 0u) : idesc_mxf4(2 * kMmaM, kTok, 2u), t_a, t_b,
                       (i != 0 || j != 0) ? 1u : 0u, one);
            }
            if (j == 3) commit_pair(bar_half + 8u * s, both, one);
          }
          commit_pair(bar_done + 8u * s, both, one);
          // (the next stage is waited for while these are under way)
          if (i + 1 < t.steps) ok = landed(i + 1);
        }
        commit_pair(bar_acc, both, one);
      }
      // after a failed wait, MMAs in flight land before the pair gives up its memory
      if (!ok) drain_wait(bar_acc, (turn - 1u) & 1u, kDrainNs);
    }
    __syncwarp();
  } else if (warp >= kScale0 && warp < kOut0) {
    const int own = warp - kScale0;                         // and its lane quadrant
    const ScaleRing ring{s_s, tmem + ((uint32_t)(32 * own) << 16) + mx_acc_cols(kTok), dev::mapa(bar_full, leader), bar_done, stages,
                         waiter};
    // (a K tile is 8 bytes of a row, a group of them a sector where rows are whole ones)
    if (p.sectors) {
      bring_scales<kTok, true>(p, ring, tile0, step, rank, half, own, lane);
    } else {
      bring_scales<kTok, false>(p, ring, tile0, step, rank, half, own, lane);
    }
  } else if (warp >= kOut0) {
    // ---- output: warp kOut0 + w has TMEM lane quadrant w, thread = weight row
    const int quad = warp - kOut0, row = quad * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t read_of_leader = dev::mapa(bar_read, leader);
    uint32_t turn = 0u;
    for (int tile = tile0; tile < p.tile_end; tile += step, ++turn) {
      const MxTile t = MxTile::at<kTok>(p, tile, rank, half);
      const int n = t.n0 + row, live = min(kTok, p.M - t.m0);
      const float bias = p.bias && n < p.N ? __uint_as_float((uint32_t)p.bias[(long long)t.l * p.N + n] << 16) : 0.0f;
      if (!__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_acc, turn & 1u, kRoleEpiMma, (int)turn))) break;
      dev::tc_fence_after();
      const auto read = [&] {                                // the accumulator may be written again
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive_remote_relaxed(read_of_leader);
      };
      const int size = p.c_f32 ? 4 : 2;
      uint8_t* to = static_cast<uint8_t*>(p.c) + (((long long)t.l * p.M + t.m0) * p.N + n) * size;
      const long long pitch = (long long)p.N * size;
      if (split > 1) {
        for (int g = 0; g < live; g += 16) {
          uint32_t v[16];
          __syncwarp();
          load_acc16(t_row + (uint32_t)g, 0u, false, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) dev::st_shared_u32(base + (uint32_t)((g + e) * kMmaM + row) * 4u, v[e]);
        }
        read();
      } else if (p.c_f32) {
        constexpr int kPart = kTok < 64 ? kTok : 64;
#pragma unroll 1
        for (int h = 0; h < kTok; h += kPart) {
          uint32_t v[kPart / 16][16];
#pragma unroll
          for (int g = 0; g < kPart / 16; ++g) dev::tmem_ld_x16(t_row + (uint32_t)(h + 16 * g), v[g]);
          dev::tmem_wait_ld();
          if (h + kPart == kTok) read();
          if (n < p.N) {
            store_tokens<kPart>(to + h * pitch, pitch, live - h, [&](uint8_t* at, int e) {
              *reinterpret_cast<float*>(at) = __uint_as_float(v[e / 16][e % 16]) + bias;
            });
          }
          __syncwarp();
        }
      } else {
        // up to half of it before any store, two tokens a register, so that the next
        // tile's MMAs may start (16 tokens at a time held them up for 4.4 us)
        constexpr int kPart = kTok < 128 ? kTok : 128;
#pragma unroll 1
        for (int h = 0; h < kTok; h += kPart) {
          uint32_t v[kPart / 2];
#pragma unroll
          for (int g = 0; g < kPart / 16; ++g) {
            uint32_t f[16];
            dev::tmem_ld_x16(t_row + (uint32_t)(h + 16 * g), f);
            dev::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v[8 * g + e] = dev::pack_bf16x2(__uint_as_float(f[2 * e]) + bias, __uint_as_float(f[2 * e + 1]) + bias);
            }
          }
          if (h + kPart == kTok) read();
          if (n < p.N) {
            store_tokens<kPart>(to + h * pitch, pitch, live - h, [&](uint8_t* at, int e) {
              *reinterpret_cast<uint16_t*>(at) = (uint16_t)(e % 2 == 0 ? v[e / 2] & 0xFFFFu : v[e / 2] >> 16);
            });
          }
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();

  if (split > 1) {
    // this rank's slice of the tokens, a column a warp and four weight rows a lane
    const MxTile& t = tile_first;
    const int live = min(kTok, p.M - t.m0);
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
    const int c0 = live * rank / split, c1 = live * (rank + 1) / split;
    const int r4 = 4 * lane;
    for (int col = c0 + warp; col < c1; col += kMxThreads / 32) {
      float v[4];
      for (int r = 0; r < split; ++r) {
        float part[4];
        dev::ld_cluster_f32x4(dev::mapa(base + (uint32_t)(col * kMmaM + r4) * 4u, (uint32_t)(2 * r + half)), part);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = r == 0 ? part[e] : v[e] + part[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int nn = t.n0 + r4 + e;
        if (nn >= p.N) continue;
        const float b = p.bias ? __uint_as_float((uint32_t)p.bias[(long long)t.l * p.N + nn] << 16) : 0.0f;
        store_mx(p, ((long long)t.l * p.M + t.m0 + col) * p.N + nn, p.bias ? v[e] + b : v[e]);
      }
    }
  }

  // ---- teardown.  After a failed wait, copies in flight land (for a bounded time)
  // before the pair gives up its memory: the leader sees both CTAs' copies, and the
  // other one leaves only after it.
  if (threadIdx.x == 0 && half == 0 && dev::ld_shared_u32(slot_abort) != 0u) {
    for (int s = 0; s < issued && s < stages; ++s) {
      drain_wait(bar_full + 8u * s, (uint32_t)(((issued - 1 - s) / stages) & 1), kDrainNs);
    }
  }
  // No CTA leaves, or frees tensor memory, while another of the cluster may still read
  // its shared memory, arrive on its barriers or run MMAs on it.
  dev::tc_fence_before();
  __syncwarp();
  dev::cluster_arrive_release();
  dev::cluster_wait_acquire();
  if (warp == 2) {
    dev::tc_fence_after();
    tmem_dealloc_pair(tmem, p.tmem_cols);
  }
}

// ---------------------------------------------------------------- launch
// How a product runs: tiles of 256 weight rows by `tokens`, counted tokens first,
// then rows, then batches; the first `whole` of them on pairs of CTAs that take one
// after another, the others on `split` pairs each.
struct MxPlan {
  int tokens;
  int whole;
  int split;
};
struct MxRing {
  int stages;
  uint32_t tmem_cols;
  size_t smem;
};

constexpr int kTokens[] = {16, 32, 64, 128, 256};

// Shared memory of a CTA, at least its share of tensor memory in the SM's: CTAs
// that fit one SM by shared memory, of whatever kernels, never wait for each
// other's columns.
size_t mx_smem(int tok, int stages, int split, uint32_t cols, const DeviceSize& dev) {
  const size_t own = (size_t)kAlignSlack + mx_bars_at(tok, stages, split) + kMxBarBytes;
  return std::max(own, std::min(dev.smem_per_sm * cols / 512, dev.smem_optin));
}

// The ring for CTAs of `steps` stages' shares of K (of all their tiles).
// For few tokens 4 stages, or 3 where nearly all pairs work (bytes in flight beyond some
// 16 MB no longer help: 64x7168x16384 on 56 pairs 16.1 us with 3 and 15.6 with 4,
// 1x7168x2048 on 28 4.9 and 4.8, but 1x18432x7168 on 72 14.3 and 14.8).
MxRing ring_of(int tokens, int split, long long pairs, long long steps, const DeviceSize& dev) {
  int stages = (int)std::min<long long>(steps, tokens <= 64 && pairs * 5 > dev.num_sms * 2 ? 3 : kMxStages);
  for (;; --stages) {
    const uint32_t cols = pow2_at_least(mx_acc_cols(tokens) + (uint32_t)(stages * kSub) * scale_cols(tokens));
    const size_t smem = mx_smem(tokens, stages, split, cols, dev);
    if (stages == 1 || (cols <= 512u && smem <= dev.smem_optin)) return MxRing{stages, cols, smem};
  }
}

void* kernel_of(int tokens) {
  switch (tokens) {
    case 16: return (void*)mx4_kernel<16>;
    case 32: return (void*)mx4_kernel<32>;
    case 64: return (void*)mx4_kernel<64>;
    case 128: return (void*)mx4_kernel<128>;
    default: return (void*)mx4_kernel<256>;
  }
}

cudaError_t read_and_clear_fault_mx4(int* out_words) {
  cudaError_t e = cudaMemcpyFromSymbol(out_words, g_fault, sizeof(int) * kFaultWords);
  if (e != cudaSuccess) return e;
  int zeros[kFaultWords] = {0};
  return cudaMemcpyToSymbol(g_fault, zeros, sizeof(zeros));
}

// Clusters of 1, 2, 3 and 4 pairs resident at once, a CTA an SM.
struct MxDevice {
  bool ready;
  int clusters[kMaxSplit];
};

// The current device's kernels, prepared at their first use.
int prepare_mx4(const DeviceSize& dev, MxDevice* out) {
  static std::mutex mu;
  static MxDevice devices[kMaxDevices] = {};
  std::lock_guard<std::mutex> lock(mu);
  MxDevice& d = devices[dev.device];
  if (!d.ready) {
    cudaError_t e = cudaSuccess;
    for (int t : kTokens) {
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel_of(t), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dev.smem_optin);
    }
    for (int i = 0; e == cudaSuccess && i < kMaxSplit; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2u * (i + 1));
      cfg.blockDim = dim3(kMxThreads);
      cfg.dynamicSmemBytes = dev.smem_optin;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2u * (i + 1);
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&d.clusters[i], kernel_of(256), &cfg);
    }
    if (e != cudaSuccess) {
      cudaGetLastError();
      return SPLITK_ERR_CUDA;
    }
    add_fault_reader(dev.device, read_and_clear_fault_mx4);
    d.ready = true;
  }
  *out = d;
  return SPLITK_OK;
}

// What a launch of `tiles` tiles costs, in microseconds: a pair's time for a K tile where
// nothing but its own work bounds it, no less than the pairs at work take to read theirs
// (6.2 bytes a picosecond: what these kernels reach on codes and scales from memory; the
// `m_tiles` tiles of the same weights read them once),
// and what comes before, between and after the tiles (for a tile in shares, their sums
// too: with its tokens). Measured, with the choice it
// decides (us): 1000x7168x16384 by 128 tokens 52.9, by 256 47.8; 2048x18432x7168
// 108.5 and 88.7; 2048x7168x2048 17.9 and 16.8; 1x7168x2048 on one pair a tile 4.8, on
// two 5.3; 16x4096x7168 10.0, 7.6, on three 7.5; 64x7168x16384 20.6 and 15.6;
// 1x500x16384 18.4, 11.1, 8.8, on four 7.1; 64x18432x7168 14.7 and 21.8 (two rounds);
// 300x10300x8192 by 128 tokens 21.9, by 256 27.7; 520x7168x4096 14.0 and 17.8;
// 16x20480x16384 in two rounds 44.8, its last 4 tiles on four pairs each 36.9.
double launch_us(long long tiles, int m_tiles, int tokens, int k_tiles, int split, bool sectors, const MxDevice& d) {
  const int fit = d.clusters[split - 1];
  if (tiles == 0) return 0.0;
  if (fit <= 0 || split > (k_tiles + kSub - 1) / kSub) return 1e30;
  // (scales that are no sectors: 0.13 to 0.18 more)
  const double own = (tokens == 256 ? 0.345 : tokens == 128 ? 0.25 : 0.22) + (sectors ? 0.0 : 0.16);
  const auto round = [&](long long n) {
    const double pairs = (double)(n * split);
    const double arrival = tokens == 256 ? 0.0 : pairs / m_tiles * (2 * kMmaM * kTileK * 17 / 32) / 6.2e6;
    return std::max(own, arrival) * ((k_tiles + split - 1) / split) + (split > 1 ? 2.7 + 0.02 * (pairs + tokens) : 0.5);
  };
  return (double)(tiles / fit) * round(fit) + (tiles % fit > 0 ? round(tiles % fit) : 0.0) + (split > 1 ? 0.0 : 2.3 + 0.01 * tokens);
}

MxPlan plan_mx4(int M, int N, int K, int L, bool sectors, const MxDevice& d) {
  const int k_tiles = (K + kTileK - 1) / kTileK;
  MxPlan best{};
  double least = 1e30;
  for (int tokens : kTokens) {
    if (tokens < 128 && tokens < M) continue;          // the smallest that holds M, or 128 or 256
    if (tokens > 16 && tokens / 2 >= M) continue;
    const int m_tiles = (M + tokens - 1) / tokens;
    const long long tiles = (long long)m_tiles * ((N + 2 * kMmaM - 1) / (2 * kMmaM)) * L;
    const double all = launch_us(tiles, m_tiles, tokens, k_tiles, 1, sectors, d);
    if (all < least) least = all, best = MxPlan{tokens, (int)tiles, 1};
    const long long rounds = d.clusters[0] > 0 ? tiles / d.clusters[0] : 0;
    for (int split = 2; split <= kMaxSplit; ++split) {
      for (long long whole : {0ll, rounds * d.clusters[0]}) {
        // (what is split has to be worth more than the estimate's errors of short K)
        const double us = launch_us(whole, m_tiles, tokens, k_tiles, 1, sectors, d) +
                          launch_us(tiles - whole, m_tiles, tokens, k_tiles, split, sectors, d);
        if (us + 0.27 < least) least = us, best = MxPlan{tokens, (int)whole, split};
      }
    }
  }
  return best;
}

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

template <int kTok>
cudaError_t launch_mx4(const uint8_t* a, const uint8_t* b, const MxParams& p, const MxPlan& plan, const DeviceSize& dev,
                       const MxDevice& d, cudaStream_t stream) {
  CUtensorMap a_map, b_map;
  if (!encode_codes(&a_map, a, p.K / 2, p.N, p.L, kMmaM) || !encode_codes(&b_map, b, p.K / 2, p.M, p.L, kTok / 2)) {
    return cudaErrorInvalidValue;
  }
  const long long tiles = (long long)((p.M + kTok - 1) / kTok) * ((p.N + 2 * kMmaM - 1) / (2 * kMmaM)) * p.L;
  const int total = (p.K + kTileK * kSub - 1) / (kTileK * kSub);
  const auto launch = [&](int first, long long end, int split, long long clusters) {
    const long long steps = (long long)((total + split - 1) / split) * ((end - first + clusters - 1) / clusters);
    const MxRing ring = ring_of(kTok, split, clusters * split, steps, dev);
    MxParams q = p;
    q.split = split, q.stages = ring.stages, q.tmem_cols = ring.tmem_cols;
    q.tile0 = first, q.tile_end = (int)end;
    return launch_chained(mx4_kernel<kTok>, dim3((unsigned)(clusters * 2 * split)), dim3(kMxThreads), ring.smem,
                          (unsigned)(2 * split), stream, a_map, b_map, q);
  };
  if (plan.whole > 0) {
    const cudaError_t e = launch(0, plan.whole, 1, std::min(plan.whole, d.clusters[0]));
    if (e != cudaSuccess) return e;
  }
  return plan.whole < tiles ? launch(plan.whole, tiles, plan.split, tiles - plan.whole) : cudaSuccess;
}

}  // namespace

}  // namespace splitk

using namespace splitk;

extern "C" {

SPLITK_API int splitk_gemm_mx4(const void* a_q, const void* a_scale, const void* b_q, const void* b_scale, const void* bias,
                               void* c, int c_type, int M, int N, int K, int L, splitk_stream_t stream) {
  if (!a_q || !a_scale || !b_q || !b_scale || !c) return SPLITK_ERR_NULL;
  if (c_type != SPLITK_DTYPE_BF16 && c_type != SPLITK_DTYPE_F32) return SPLITK_ERR_INVALID_ARGUMENT;
  if (M < 1 || N < 1 || K < 1 || L < 1 || K % kMxBlock != 0 || L > 65535 || N > 65535 * 128 || K > (1 << 30) || M > (1 << 30)) {
    return SPLITK_ERR_INVALID_SHAPE;
  }
  // a launch's CTAs: eight for each 16 tokens by 256 weight rows at most
  if (((long long)M + 15) / 16 * ((N + 255) / 256) * L > (1ll << 27)) return SPLITK_ERR_INVALID_SHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(bias, 2) || !aligned(c, c_type == SPLITK_DTYPE_F32 ? 4u : 2u)) {
    return SPLITK_ERR_MISALIGNED;
  }
  DeviceSize dev;
  int rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  MxDevice d;
  rc = prepare_mx4(dev, &d);
  if (rc != SPLITK_OK) return rc;
  const int blocks = K / kMxBlock;
  const bool sectors = blocks % 32 == 0 && aligned(a_scale, 32) && aligned(b_scale, 32);
  const MxPlan plan = plan_mx4(M, N, K, L, sectors, d);
  if (plan.tokens == 0) return SPLITK_ERR_NO_FIT;      // no CTA pair of it fits the device
  // (a CTA counts the K tiles of all its tiles)
  if (((long long)plan.whole / std::max(d.clusters[0], 1) + 1) * ((K + kTileK - 1) / kTileK) > (1ll << 30)) {
    return SPLITK_ERR_INVALID_SHAPE;
  }
  const MxParams p{static_cast<const uint8_t*>(a_scale), static_cast<const uint8_t*>(b_scale),
                   static_cast<const uint16_t*>(bias), c, c_type == SPLITK_DTYPE_F32, M, N, K, L, 1, 1, 0, 0, 0u, sectors,
                   wait_limit_ns(), injected()};
  const uint8_t *a = static_cast<const uint8_t*>(a_q), *b = static_cast<const uint8_t*>(b_q);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (plan.tokens) {
    case 16: return launched(launch_mx4<16>(a, b, p, plan, dev, d, s));
    case 32: return launched(launch_mx4<32>(a, b, p, plan, dev, d, s));
    case 64: return launched(launch_mx4<64>(a, b, p, plan, dev, d, s));
    case 128: return launched(launch_mx4<128>(a, b, p, plan, dev, d, s));
    default: return launched(launch_mx4<256>(a, b, p, plan, dev, d, s));
  }
}

}  // extern "C"
