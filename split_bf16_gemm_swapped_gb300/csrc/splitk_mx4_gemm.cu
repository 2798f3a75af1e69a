// splitk_gemm_mx4(): the matrix product of two operands in microscaled 4-bit codes
// (splitk_mx4.cuh) on the tensor cores' own instruction for them: E2M1 codes and
// E8M0 scales go in as they are, nothing is converted.
//
// A CTA owns 128 weight rows (the MMA's M side) and kTok tokens (its N side).  TMA
// brings codes, 256 of K wide, from both operands into a ring of shared memory
// (K-major, 128-byte swizzle).  Scale warps bring the tiles' scales into shared
// memory in the order that a copy into tensor memory wants: for 128 rows and four
// blocks of K, 512 bytes, row r's four codes at 16 (r % 32) + 4 (r / 32).  The
// issuing thread copies them (tcgen05.cp, to all four lane quadrants) into columns
// of the tile's own and issues four MMAs of K = 64.
//
// `split` CTAs of a cluster may share one output tile, each taking a contiguous
// run of K tiles; each leaves its f32 sums in its own shared memory and then adds
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

constexpr int kMxThreads = 256;
constexpr int kScale0 = 4, kScaleWarps = 4;          // the warps that bring scales (and store the output)
constexpr int kTileK = 256;                          // codes of a K tile: 128 bytes
constexpr int kMxStages = 10;                        // at most
constexpr uint32_t kCodesA = kMmaM * (kTileK / 2);   // 16 KiB
constexpr uint32_t kScaleAtom = 512;                 // 128 rows x 4 scales
constexpr uint32_t kMxBarBytes = 512;
constexpr int kMaxSplit = 8;

__host__ __device__ constexpr uint32_t codes_b(int tok) { return (uint32_t)tok * (kTileK / 2); }
__host__ __device__ constexpr int groups_b(int tok) { return (tok + 127) / 128; }     // of 128 tokens
__host__ __device__ constexpr uint32_t scales_of(int tok) { return 2u * kScaleAtom * (1u + groups_b(tok)); }
__host__ __device__ constexpr uint32_t stage_bytes(int tok) { return kCodesA + codes_b(tok) + scales_of(tok); }
__host__ __device__ constexpr uint32_t mx_acc_cols(int tok) { return tok < 32 ? 32u : (uint32_t)tok; }
__host__ __device__ constexpr uint32_t scale_cols(int tok) { return 8u * (1u + groups_b(tok)); }   // of a stage

// kind::mxf4: E2M1 operands, both K-major, E8M0 scales for each 32, f32 accumulator;
// the scales of a K = 64 step are the lower (id 0) or upper (id 2) half of a word.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27) | (id << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scale,
                                         uint32_t b_scale, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
      : "memory");
}

// 32 rows of 16 bytes (unswizzled) into four columns of each lane quadrant.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t s_desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(s_desc) : "memory");
}

// Shared-memory descriptor of such rows: no swizzle, eight rows (128 bytes) apart.
__device__ __forceinline__ uint64_t smem_desc_rows16(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(16u >> 4) << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

struct MxParams {
  const uint8_t* a_scale;   // [L][N][K / 32]
  const uint8_t* b_scale;   // [L][M][K / 32]
  const uint16_t* bias;     // bf16 [L][N], or null
  void* c;                  // bf16 or f32 [L][M][N]
  bool c_f32;
  int M, N, K, L;
  int split, stages;
  uint32_t tmem_cols;
  int a_align, b_align;     // of the scales' rows: 8, 4 or 1 bytes
  unsigned long long limit_ns;
  unsigned inject;
};

// The scale codes of 8 blocks of K of one row (two words of four), 127 past K.
__device__ __forceinline__ uint2 load_scales(const uint8_t* row, int at, int blocks, int align) {
  constexpr uint32_t kOnes = 0x7F7F7F7Fu;
  if (align == 8) return *reinterpret_cast<const uint2*>(row + at);       // (blocks a multiple of 8)
  if (align == 4) {
    return make_uint2(*reinterpret_cast<const uint32_t*>(row + at),
                      at + 4 < blocks ? *reinterpret_cast<const uint32_t*>(row + at + 4) : kOnes);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i / 4] |= (at + i < blocks ? (uint32_t)row[at + i] : 127u) << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}

// One output from its sum.
__device__ __forceinline__ void store_mx(const MxParams& p, long long at, float v) {
  if (p.c_f32) {
    static_cast<float*>(p.c)[at] = v;
  } else {
    static_cast<uint16_t*>(p.c)[at] = (uint16_t)dev::pack_bf16x2(v, 0.0f);
  }
}

template <int kTok>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx4_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map, const MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (dev::smem_u32(smem_raw) + (kAlignSlack - 1)) & ~(kAlignSlack - 1);
  const int stages = p.stages, split = p.split;
  const uint32_t s_a = base;
  const uint32_t s_b = s_a + (uint32_t)stages * kCodesA;
  const uint32_t s_s = s_b + (uint32_t)stages * codes_b(kTok);
  const uint32_t s_bar = s_s + (uint32_t)stages * scales_of(kTok);
  const uint32_t bar_full = s_bar;                          // [kMxStages] the codes landed
  const uint32_t bar_scale = s_bar + 8u * kMxStages;        // [kMxStages] the scales are there
  const uint32_t bar_free = s_bar + 16u * kMxStages;        // [kMxStages] the MMAs have read both
  const uint32_t bar_acc = s_bar + 24u * kMxStages;         // the accumulator is complete
  const uint32_t slot_tmem = bar_acc + 8u, slot_abort = bar_acc + 12u;

  const int warp = (int)(threadIdx.x >> 5), lane = (int)(threadIdx.x & 31);
  const int rank = split > 1 ? (int)dev::cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / split;
  const int m_tiles = (p.M + kTok - 1) / kTok, n_tiles = (p.N + kMmaM - 1) / kMmaM;
  const int m0 = (tile % m_tiles) * kTok, l = tile / m_tiles / n_tiles, n0 = (tile / m_tiles % n_tiles) * kMmaM;
  const int total = (p.K + kTileK - 1) / kTileK;
  const int each = total / split, extra = total % split;
  const int k_tiles = each + (rank < extra ? 1 : 0);
  const int kt0 = rank * each + (rank < extra ? rank : extra);
  const Waiter waiter{slot_abort, p.limit_ns};

  if (warp == 3 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      dev::mbar_init(bar_full + 8u * s, 1u);
      dev::mbar_init(bar_scale + 8u * s, 1u);
      dev::mbar_init(bar_free + 8u * s, 1u);
    }
    dev::mbar_init(bar_acc, 1u);
    dev::st_shared_u32(slot_abort, 0u);
    dev::fence_barrier_init();
  } else if (warp == 2) {
    dev::tmem_alloc(slot_tmem, p.tmem_cols);
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
  // While the work ahead in the stream completes, the ring's first weight tiles come
  // to L2 (which is where a kernel's writes would change them: nothing is read early).
  if (warp == 0 && lane < min(stages, k_tiles)) dev::tma_prefetch_3d(&a_map, (kt0 + lane) * (kTileK / 2), n0, l);
  dev::griddep_wait();
  const uint32_t tmem = dev::ld_shared_u32(slot_tmem);

  const int live = min(kTok, p.M - m0);
  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      const uint64_t stream_once = dev::policy_evict_first(), keep = dev::policy_evict_normal();
      const uint64_t policy_a = m_tiles == 1 ? stream_once : keep;
      RingPos pos{0, 0u};
      for (int kt = 0; kt < k_tiles; ++kt, pos.advance(1, stages)) {
        const uint32_t s = (uint32_t)pos.index;
        if (kt >= stages && !waiter.wait<false>(bar_free + 8u * s, pos.phase ^ 1u, kRoleWeightTma, kt)) break;
        dev::mbar_arrive_expect_tx(bar_full + 8u * s, kCodesA + codes_b(kTok));
        dev::tma_load_3d_hint(s_a + s * kCodesA, &a_map, (kt0 + kt) * (kTileK / 2), n0, l, bar_full + 8u * s, policy_a);
        dev::tma_load_3d_hint(s_b + s * codes_b(kTok), &b_map, (kt0 + kt) * (kTileK / 2), m0, l, bar_full + 8u * s, keep);
        ++issued;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      RingPos pos{0, 0u};
      const uint64_t a_desc = dev::smem_desc_sw128(s_a), b_desc = dev::smem_desc_sw128(s_b);
      const uint64_t s_desc = smem_desc_rows16(s_s);
      for (int kt = 0; kt < k_tiles; ++kt, pos.advance(1, stages)) {
        const uint32_t s = (uint32_t)pos.index;
        if (!waiter.wait<false>(bar_scale + 8u * s, pos.phase, kRoleMma, kt)) break;
        const uint32_t t_a = tmem + mx_acc_cols(kTok) + s * scale_cols(kTok), t_b = t_a + 8u;
        dev::tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2 * (1 + groups_b(kTok)); ++i) {
          tmem_cp_scales(t_a + 4u * i, dev::smem_desc_advance(s_desc, s * scales_of(kTok) + kScaleAtom * i));
        }
        if (!waiter.wait<false>(bar_full + 8u * s, pos.phase, kRoleMma, kt)) break;
        const uint64_t a_d = dev::smem_desc_advance(a_desc, s * kCodesA), b_d = dev::smem_desc_advance(b_desc, s * codes_b(kTok));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma_mxf4(tmem, dev::smem_desc_advance(a_d, 32u * j), dev::smem_desc_advance(b_d, 32u * j),
                   j % 2 == 0 ? idesc_mxf4(kMmaM, kTok, 0u) : idesc_mxf4(kMmaM, kTok, 2u), t_a + 4u * (j / 2),
                   t_b + 4u * groups_b(kTok) * (j / 2), (kt != 0 || j != 0) ? 1u : 0u);
        }
        dev::mma_commit(bar_free + 8u * s);
      }
      dev::mma_commit(bar_acc);
    }
    __syncwarp();
  } else if (warp >= kScale0) {
    // A lane has rows lane + 32 g of each group of 128: for each word of K their four
    // scales lie side by side, one 16-byte store.  A warp takes every kScaleWarps-th
    // K tile; its loads are under way while it waits for the slot.
    const int blocks = p.K / kMxBlock;
    const uint8_t* a_rows = p.a_scale + (long long)l * p.N * blocks;
    const uint8_t* b_rows = p.b_scale + (long long)l * p.M * blocks;
    RingPos pos = RingPos::at(warp - kScale0, stages);
    for (int kt = warp - kScale0; kt < k_tiles; kt += kScaleWarps) {
      const uint32_t s = (uint32_t)pos.index;
      const int at = (kt0 + kt) * (kTileK / kMxBlock);
      uint2 a[4], b[groups_b(kTok)][4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + lane + 32 * g;
        a[g] = n < p.N ? load_scales(a_rows + (long long)n * blocks, at, blocks, p.a_align) : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int q = 0; q < groups_b(kTok); ++q) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int m = m0 + 128 * q + lane + 32 * g;
          const bool in = 128 * q + 32 * g < kTok && m < p.M;
          b[q][g] = in ? load_scales(b_rows + (long long)m * blocks, at, blocks, p.b_align) : make_uint2(0u, 0u);
        }
      }
      if (kt >= stages &&
          !__all_sync(0xFFFFFFFFu, waiter.wait<false>(bar_free + 8u * s, pos.phase ^ 1u, kRoleEpiDecode, kt))) break;
      const uint32_t dst = s_s + s * scales_of(kTok) + 16u * lane;
      dev::st_shared_v4(dst, a[0].x, a[1].x, a[2].x, a[3].x);
      dev::st_shared_v4(dst + kScaleAtom, a[0].y, a[1].y, a[2].y, a[3].y);
#pragma unroll
      for (int q = 0; q < groups_b(kTok); ++q) {
        dev::st_shared_v4(dst + (2u + q) * kScaleAtom, b[q][0].x, b[q][1].x, b[q][2].x, b[q][3].x);
        dev::st_shared_v4(dst + (2u + groups_b(kTok) + q) * kScaleAtom, b[q][0].y, b[q][1].y, b[q][2].y, b[q][3].y);
      }
      dev::fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0 && (p.inject & kInjectSkipPublish) == 0) dev::mbar_arrive(bar_scale + 8u * s);
      for (int i = 0; i < kScaleWarps; ++i) pos.advance(1, stages);
    }
  }

  // ---- epilogue: a warp a TMEM lane quadrant, thread = weight row
  const int row = (warp & 3) * 32 + lane, n = n0 + row;
  waiter.wait<false>(bar_acc, 0u, kRoleEpiMma, 0);
  __syncthreads();
  dev::tc_fence_after();
  if (warp >= kScale0) {
    const float bias = p.bias && n < p.N ? __uint_as_float((uint32_t)p.bias[(long long)l * p.N + n] << 16) : 0.0f;
    const uint32_t t_row = tmem + ((uint32_t)(row & ~31) << 16);
    for (int g = 0; g * 16 < live; ++g) {
      uint32_t v[16];
      __syncwarp();
      if (kTok < 16) {
        uint32_t u[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          dev::tmem_ld_x4(t_row + 4u * q, u[0], u[1], u[2], u[3]);
          dev::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] = u[e], v[8 + 4 * q + e] = 0u;
        }
      } else {
        load_acc16(t_row + 16u * g, 0u, false, v);
      }
      const int cols = min(16, live - g * 16);
      if (split > 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (e < cols) dev::st_shared_u32(base + (uint32_t)((g * 16 + e) * kMmaM + row) * 4u, v[e]);
        }
      } else if (n < p.N) {
        const long long at = ((long long)l * p.M + m0 + g * 16) * p.N + n;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (e < cols) store_mx(p, at + (long long)e * p.N, p.bias ? __uint_as_float(v[e]) + bias : __uint_as_float(v[e]));
        }
      }
    }
  }
  if (split > 1) {
    // this rank's slice of the tokens, a column a warp and four weight rows a lane
    __syncwarp();
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
    const int c0 = live * rank / split, c1 = live * (rank + 1) / split;
    const int r4 = 4 * lane;
    for (int col = c0 + warp; col < c1; col += kMxThreads / 32) {
      float v[4];
      for (int r = 0; r < split; ++r) {
        float part[4];
        dev::ld_cluster_f32x4(dev::mapa(base + (uint32_t)(col * kMmaM + r4) * 4u, (uint32_t)r), part);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = r == 0 ? part[e] : v[e] + part[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int nn = n0 + r4 + e;
        if (nn >= p.N) continue;
        const float b = p.bias ? __uint_as_float((uint32_t)p.bias[(long long)l * p.N + nn] << 16) : 0.0f;
        store_mx(p, ((long long)l * p.M + m0 + col) * p.N + nn, p.bias ? v[e] + b : v[e]);
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
  // No CTA leaves while another of the cluster may still read its shared memory.
  dev::tc_fence_before();
  __syncwarp();
  if (split > 1) {
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
  } else {
    __syncthreads();
  }
  if (warp == 2) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ---------------------------------------------------------------- launch
struct MxPlan {
  int tokens, split, stages;
  uint32_t tmem_cols;
  size_t smem;
};

constexpr int kTokens[] = {8, 16, 32, 64, 128, 256};

// Shared memory of a CTA, at least its share of tensor memory in the SM's: CTAs
// that fit one SM by shared memory, of whatever kernels, never wait for each
// other's columns.
size_t mx_smem(int tok, int stages, int split, uint32_t cols, const DeviceSize& dev) {
  const size_t ring = (size_t)kAlignSlack + (size_t)stages * stage_bytes(tok) + kMxBarBytes;
  const size_t sums = split > 1 ? (size_t)kAlignSlack + (size_t)tok * kMmaM * 4 : 0;
  return std::max(std::max(ring, sums), std::min(dev.smem_per_sm * cols / 512, dev.smem_optin));
}

bool make_plan(int tokens, int split, int k_tiles, const DeviceSize& dev, MxPlan* out) {
  const int mine = (k_tiles + split - 1) / split;
  for (int stages = std::min(mine, kMxStages); stages >= 1; --stages) {
    const uint32_t cols = pow2_at_least(mx_acc_cols(tokens) + (uint32_t)stages * scale_cols(tokens));
    if (cols > 512u) continue;
    const size_t smem = mx_smem(tokens, stages, split, cols, dev);
    if (smem > dev.smem_optin) continue;
    *out = MxPlan{tokens, split, stages, cols, smem};
    return true;
  }
  return false;
}

void* kernel_of(int tokens) {
  switch (tokens) {
    case 8: return (void*)mx4_kernel<8>;
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

// The current device's kernels, prepared at their first use.
int prepare_mx4(int device, const DeviceSize& dev) {
  static std::mutex mu;
  static bool ready[kMaxDevices] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (ready[device]) return SPLITK_OK;
  for (int t : kTokens) {
    if (cudaFuncSetAttribute(kernel_of(t), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dev.smem_optin) != cudaSuccess) {
      cudaGetLastError();
      return SPLITK_ERR_CUDA;
    }
  }
  add_fault_reader(device, read_and_clear_fault_mx4);
  ready[device] = true;
  return SPLITK_OK;
}

MxPlan plan_mx4(int M, int N, int K, int L, const DeviceSize& dev) {
  const int k_tiles = (K + kTileK - 1) / kTileK;
  int tokens = 256;
  for (int t : {128, 64, 32, 16, 8}) {
    if (t >= M) tokens = t;
  }
  const long long tiles = (long long)((M + tokens - 1) / tokens) * ((N + kMmaM - 1) / kMmaM) * L;
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= 2 * dev.num_sms && split * 2 <= k_tiles) split *= 2;
  MxPlan best{};
  for (; split >= 1; --split) {
    if (make_plan(tokens, split, k_tiles, dev, &best)) return best;
  }
  return best;
}

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

template <int kTok>
cudaError_t launch_mx4(const uint8_t* a, const uint8_t* b, const MxParams& p, const MxPlan& plan, cudaStream_t stream) {
  CUtensorMap a_map, b_map;
  if (!encode_codes(&a_map, a, p.K / 2, p.N, p.L, kMmaM) || !encode_codes(&b_map, b, p.K / 2, p.M, p.L, kTok)) {
    return cudaErrorInvalidValue;
  }
  const long long tiles = (long long)((p.M + kTok - 1) / kTok) * ((p.N + kMmaM - 1) / kMmaM) * p.L;
  return launch_chained(mx4_kernel<kTok>, dim3((unsigned)(tiles * plan.split)), dim3(kMxThreads), plan.smem,
                        (unsigned)plan.split, stream, a_map, b_map, p);
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
  // a launch's CTAs: eight for each 8 tokens by 128 weight rows at most
  if (((long long)M + 7) / 8 * ((N + 127) / 128) * L > (1ll << 27)) return SPLITK_ERR_INVALID_SHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(bias, 2) || !aligned(c, c_type == SPLITK_DTYPE_F32 ? 4u : 2u)) {
    return SPLITK_ERR_MISALIGNED;
  }
  DeviceSize dev;
  int rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  rc = prepare_mx4(dev.device, dev);
  if (rc != SPLITK_OK) return rc;
  const MxPlan plan = plan_mx4(M, N, K, L, dev);
  if (plan.tokens == 0) return SPLITK_ERR_NO_FIT;
  const int blocks = K / kMxBlock;
  const auto align = [&](const void* s) { return blocks % 8 == 0 && aligned(s, 8) ? 8 : blocks % 4 == 0 && aligned(s, 4) ? 4 : 1; };
  const MxParams p{static_cast<const uint8_t*>(a_scale), static_cast<const uint8_t*>(b_scale),
                   static_cast<const uint16_t*>(bias), c, c_type == SPLITK_DTYPE_F32, M, N, K, L, plan.split, plan.stages,
                   plan.tmem_cols, align(a_scale), align(b_scale), wait_limit_ns(), injected()};
  const uint8_t *a = static_cast<const uint8_t*>(a_q), *b = static_cast<const uint8_t*>(b_q);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (plan.tokens) {
    case 8: return launched(launch_mx4<8>(a, b, p, plan, s));
    case 16: return launched(launch_mx4<16>(a, b, p, plan, s));
    case 32: return launched(launch_mx4<32>(a, b, p, plan, s));
    case 64: return launched(launch_mx4<64>(a, b, p, plan, s));
    case 128: return launched(launch_mx4<128>(a, b, p, plan, s));
    default: return launched(launch_mx4<256>(a, b, p, plan, s));
  }
}

}  // extern "C"
