// Log probabilities of a vocabulary's logits: splitk_logprobs().
//
// For a row x of V logits, with m = max x:
//   S = sum exp(x - m),  T = sum exp(x - m) (x - m)
//   logprob(i) = x[i] - m - log S,   entropy = log S - T / S
// and the k largest logits, equal ones by the lowest index.
//
// One pass reads the row.  A warp takes 256 consecutive logits (a group) at a
// time and keeps a running maximum with S and T rescaled when it grows; the
// group's maximum, needed for that anyway, is also written down.  If at least k
// groups' maxima reach a bound, the k best logits are in groups whose maxima do
// (a logit of any other group has k larger ones); and the k best groups by
// (maximum, lowest index) hold them too.  So only some k groups are read a
// second time, and where fewer logits than k are above the bound, some that equal
// it, from the row's start.
//
// Memory bounds the pass (1024 x 131072 bf16: 46 us without alternatives, 87 % of
// the copy rate); each row's join and selection is what 20 alternatives add (6 us of
// a launch: 52), as it overlaps only with other rows' passes.  Rows of
// a few thousand logits are bound by the instructions of either (4096 x 8000: 19
// us and 35, the copy rate 10).
//
// A cluster of CTAs shares a row when there are few rows; the first CTA then
// reads the others' sums and maxima from their shared memory.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"
#include "splitk_device.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

constexpr int kGroup = 256;                 // logits of a group: eight of each lane
constexpr int kMaxTop = 32;
constexpr int kMaxVocab = 1 << 22;
constexpr int kMaxGroups = 64;              // groups read a second time
constexpr int kMaxCandidates = 1024;        // logits of theirs that may be among the top
constexpr int kFewCandidates = 128;         // that many are ranked by counting
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kFarBelow = -1000.0f;       // in powers of two: exp is 0, and so is exp times it
constexpr uint32_t kFull = 0xFFFFFFFFu;

struct LogprobParams {
  const void* x;             // [rows][stride]
  long long stride;
  const long long* tokens;   // [rows], or null
  float* logprob;            // [rows], or null
  float* entropy;            // [rows]
  long long* top_ids;        // [rows][k], or null
  float* top_logprobs;       // [rows][k], or null
  int rows, V, k;
};

// kType: 1 bf16, 2 f32, 3 f16.  A lane's eight logits of a group come in kLoads
// 16-byte words, kAhead groups at a time; the largest of them is found on the
// packed values.
__device__ __forceinline__ float f16_one(uint16_t v) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(v));
  return f;
}
template <int kType>
struct Logit;
template <>
struct Logit<1> {
  static constexpr int kPerLoad = 8, kLoads = 1, kAhead = 4;
  static constexpr float kNear = 65536.0f, kLowest = -3.38953139e38f;
  __device__ static uint32_t pair_of(float v) { return dev::pack_bf16x2(v, v); }
  using T = uint16_t;
  __device__ static float one(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  __device__ static uint32_t pair_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // the words with no logit under `low` (a pair); a NaN stays one
  __device__ static void raise(uint4 (&w)[1], uint32_t low) {
    uint32_t* u[4] = {&w[0].x, &w[0].y, &w[0].z, &w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(*u[i]) : "r"(low));
  }
  __device__ static float max_of(const uint4 (&w)[1]) {
    const uint32_t m = pair_max(pair_max(w[0].x, w[0].y), pair_max(w[0].z, w[0].w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  __device__ static void unpack(const uint4 (&w)[1], float (&f)[8]) {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Logit<3> {
  static constexpr int kPerLoad = 8, kLoads = 1, kAhead = 4;
  static constexpr float kNear = 60000.0f, kLowest = -65504.0f;
  __device__ static uint32_t pair_of(float v) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(v), "f"(v));
    return d;
  }
  using T = uint16_t;
  __device__ static float one(uint16_t v) { return f16_one(v); }
  __device__ static uint32_t pair_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  // the words with no logit under `low` (a pair); a NaN stays one
  __device__ static void raise(uint4 (&w)[1], uint32_t low) {
    uint32_t* u[4] = {&w[0].x, &w[0].y, &w[0].z, &w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(*u[i]) : "r"(low));
  }
  __device__ static float max_of(const uint4 (&w)[1]) {
    const uint32_t m = pair_max(pair_max(w[0].x, w[0].y), pair_max(w[0].z, w[0].w));
    return fmaxf(f16_one((uint16_t)m), f16_one((uint16_t)(m >> 16)));
  }
  __device__ static void unpack(const uint4 (&w)[1], float (&f)[8]) {
    const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = f16_one((uint16_t)u[i]);
      f[2 * i + 1] = f16_one((uint16_t)(u[i] >> 16));
    }
  }
};
template <>
struct Logit<2> {
  static constexpr int kPerLoad = 4, kLoads = 2, kAhead = 2;
  static constexpr float kLowest = -3.402823466e38f;
  using T = float;
  __device__ static float one(float v) { return v; }
  __device__ static void unpack(const uint4 (&w)[2], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(w[i].x), f[4 * i + 1] = __uint_as_float(w[i].y);
      f[4 * i + 2] = __uint_as_float(w[i].z), f[4 * i + 3] = __uint_as_float(w[i].w);
    }
  }
  __device__ static float max_of(const uint4 (&w)[2]) {
    float f[8];
    unpack(w, f);
    return fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
  }
};

__device__ __forceinline__ float exp2_approx(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A number that orders as the logit does (-0 as 0); 0 stands below every
// logit, and a NaN above.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

// Logits of a row in their order: by value, then by the lowest index.
__device__ __forceinline__ uint64_t key_of(uint32_t order, int id) { return ((uint64_t)order << 32) | (uint32_t)~id; }
__device__ __forceinline__ long long id_of(uint64_t key) { return (long long)(uint32_t)~(uint32_t)key; }

// A row as 16-byte words: position p counts from the aligned address at or
// before the row's first logit, so logit i stands at p = i + shift.  Groups
// that reach over either end are read one logit at a time, and what is not of
// the row reads as -inf.
template <int kType>
struct Row {
  using E = Logit<kType>;
  const typename E::T* x;
  int shift, V;
  __device__ Row(const LogprobParams& p, int row)
      : x(static_cast<const typename E::T*>(p.x) + (long long)row * p.stride), V(p.V) {
    shift = (int)(((uintptr_t)x & 15u) / sizeof(typename E::T));
  }
  __device__ int groups() const { return (shift + V + kGroup - 1) / kGroup; }
  // whether groups [g, h) lie in the row
  __device__ bool inside(int g, int h) const { return g * kGroup >= shift && h * kGroup <= shift + V; }
  // position of the j-th of a lane's eight logits of group `g`
  __device__ static int at(int g, int lane, int j) {
    return g * kGroup + (j / E::kPerLoad) * 32 * E::kPerLoad + lane * E::kPerLoad + j % E::kPerLoad;
  }
  __device__ __forceinline__ void load_words(int g, int lane, uint4 (&w)[E::kLoads]) const {
#pragma unroll
    for (int i = 0; i < E::kLoads; ++i) {
      w[i] = *reinterpret_cast<const uint4*>(x + (at(g, lane, i * E::kPerLoad) - shift));
    }
  }
  __device__ __forceinline__ void load_group(int g, int lane, float (&f)[8]) const {
    if (inside(g, g + 1)) {
      uint4 w[E::kLoads];
      load_words(g, lane, w);
      E::unpack(w, f);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = at(g, lane, j) - shift;
      f[j] = i >= 0 && i < V ? E::one(x[i]) : -INFINITY;
    }
  }
};

// Sums relative to a maximum; in powers of two (d = (x - m) log2 e).
struct Sums {
  float m, s, t;
  // the same sums relative to `to` >= m
  __device__ __forceinline__ void rebase(float to) {
    if (m == -INFINITY) {                  // nothing but masked logits so far: s and t are 0 (or NaN)
      m = to;
      return;
    }
    const float d = fminf((to - m) * kLog2e, -kFarBelow), f = exp2_approx(-d);
    t = f * (t - d * s);
    s *= f;
    m = to;
  }
};

// ... of a warp, a CTA or a row.  Where one logit outweighs the others, its 1
// rounds away what little they add, and the logarithm of 1 + s wants that s: so
// the sum without the lane that holds the largest logit is kept too, and where
// that lane is (its logits can be summed again).
struct Part {
  Sums sums;
  float rest;
  int where;                 // CTA of the row << 16 | warp << 8 | lane
};

__device__ __forceinline__ float warp_max(float v) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(kFull, v, o);
    v = w > v ? w : v;
  }
  return v;
}

// One warp: the parts its lanes hold, added relative to their largest maximum.
__device__ __forceinline__ Part join(Part part) {
  const float top = warp_max(part.sums.m);
  const bool largest = part.sums.m == top;
  part.sums.rebase(top);
  part.rest = warp_sum(largest ? part.rest : part.sums.s);
  part.sums.s = warp_sum(part.sums.s);
  part.sums.t = warp_sum(part.sums.t);
  part.where = __shfl_sync(kFull, part.where, __ffs(__ballot_sync(kFull, largest)) - 1);
  return part;
}

// Adds eight logits of each lane, whose warp's largest is at most a.m; they may
// be so far below it that they are not finite beside it.
__device__ __forceinline__ void add_any(Sums& a, const float (&f)[8]) {
  const float base = a.m == -INFINITY ? 0.0f : a.m;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = max_nan((f[j] - base) * kLog2e, kFarBelow);
    const float e = exp2_approx(d);
    a.s += e;
    a.t = fmaf(e, d, a.t);
  }
}

// The same for logits at most 1000 below it, two at a time.
__device__ __forceinline__ void add_near(Sums& a, const float (&f)[8]) {
  const uint64_t minus = dev::f32x2(-a.m, -a.m), scale = dev::f32x2(kLog2e, kLog2e);
  uint64_t s = dev::f32x2(a.s, 0.0f), t = dev::f32x2(a.t, 0.0f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t d = dev::f32x2_mul(dev::f32x2_add(dev::f32x2(f[j], f[j + 1]), minus), scale);
    float d0, d1;
    dev::f32x2_split(d, d0, d1);
    const uint64_t e = dev::f32x2(exp2_approx(d0), exp2_approx(d1));
    s = dev::f32x2_add(s, e);
    t = dev::f32x2_fma(e, d, t);
  }
  float s0, s1, t0, t1;
  dev::f32x2_split(s, s0, s1);
  dev::f32x2_split(t, t0, t1);
  a.s = s0 + s1;
  a.t = t0 + t1;
}

// The same from packed words.  Of 16-bit logits two at a time are raised to 800
// under the maximum first (exp is 0 from 104 on), where the type resolves that;
// elsewhere, and for 32-bit ones, each distance is clamped.
template <int kType>
__device__ __forceinline__ void add_words(Sums& a, uint4 (&w)[Logit<kType>::kLoads]) {
  float f[8];
  if constexpr (kType != 2) {
    if (fabsf(a.m) < Logit<kType>::kNear) {
      Logit<kType>::raise(w, Logit<kType>::pair_of(a.m - 800.0f));
      Logit<kType>::unpack(w, f);
      add_near(a, f);
      return;
    }
  }
  Logit<kType>::unpack(w, f);
  add_any(a, f);
}

// One warp: the k best of the n maxima in `best` (0 where taken), by the lowest
// group where equal, as group numbers into `sel`; the last one's maximum is the
// result.  Lane l holds the maximum of the l-th 32nd of the groups.
__device__ __forceinline__ uint32_t draw_groups(uint32_t* best, int n, int k, int lane, int* sel) {
  const int span = ((n + 1023) / 1024) * 32;
  uint32_t mine = 0, last = 0;
  for (int i = 0; i < n; i += 32) {
    const uint32_t top = __reduce_max_sync(kFull, i + lane < n ? best[i + lane] : 0u);
    if (i / span == lane) mine = max(mine, top);
  }
  for (int r = 0; r < k; ++r) {
    last = __reduce_max_sync(kFull, mine);
    const int owner = __ffs(__ballot_sync(kFull, mine == last)) - 1;
    bool found = false;
    uint32_t rest = 0;
    for (int i = 0; i < span; i += 32) {
      const int g = owner * span + i + lane;
      uint32_t v = g < n ? best[g] : 0u;
      if (!found) {
        const uint32_t hit = __ballot_sync(kFull, g < n && v == last);
        if (hit != 0) {
          found = true;
          if (lane == __ffs(hit) - 1) {
            best[g] = 0;
            sel[r] = g;
            v = 0;
          }
        }
      }
      rest = max(rest, __reduce_max_sync(kFull, v));
    }
    if (lane == owner) mine = rest;
    __syncwarp();
  }
  return last;
}

// One warp: the first `need` logits of the row that equal `value`, as keys into
// `cand`; `best` holds the groups' maxima, `bound` the value's order.  Maxima pass over
// NaN, so a group whose maximum is `value` may hold nothing else of the row (where
// the value is -inf, which what is beside a row reads as): its NaN count as equal.
// That leaves no logit of the row out, and the caller has `need` of them.
template <int kType>
__device__ __noinline__ void first_equal(Row<kType> row, const uint32_t* best, int n, uint32_t bound, float value,
                                         int lane, int need, uint64_t* cand) {
  constexpr int kRun = Logit<kType>::kPerLoad;     // consecutive logits of a lane
  for (int g0 = 0; g0 < n; g0 += 32) {
    uint32_t there = __ballot_sync(kFull, g0 + lane < n && best[min(g0 + lane, n - 1)] >= bound);
    for (; there != 0; there &= there - 1) {
      const int g = g0 + __ffs(there) - 1;
      const bool nan_too = best[g] == bound;
      float f[8];
      row.load_group(g, lane, f);
#pragma unroll
      for (int h = 0; h < 8; h += kRun) {
        uint32_t equal = 0;
#pragma unroll
        for (int j = h; j < h + kRun; ++j) {
          const int id = Row<kType>::at(g, lane, j) - row.shift;
          const bool is = f[j] == value || (nan_too && f[j] != f[j]);
          if (is && id >= 0 && id < row.V) equal |= 1u << j;
        }
        int rank = __popc(equal);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int below = __shfl_up_sync(kFull, rank, o);
          rank += lane >= o ? below : 0;
        }
        const int all = __shfl_sync(kFull, rank, 31);
        rank -= __popc(equal);
        for (; equal != 0 && rank < need; equal &= equal - 1, ++rank) {
          cand[rank] = key_of(bound, Row<kType>::at(g, lane, __ffs(equal) - 1) - row.shift);
        }
        if (all >= need) return;
        need -= all;
        cand += all;
      }
    }
  }
}

// A lower bound on the k-th largest logit is the k-th largest of 32 of the lanes'
// values (logits of the row, all different ones), each warp's largest; 0 if there
// are not that many.  Of 64 where `wide`.  First each warp puts its own into `some` ...
template <int kWarps>
__device__ __forceinline__ void top_lanes(uint32_t value, bool wide, int warp, int lane, uint32_t* some) {
  const auto next = [&](int at) {
#pragma unroll
    for (int i = 0; i < 32 / kWarps; ++i) {
      const uint32_t top = __reduce_max_sync(kFull, value);
      const int owner = __ffs(__ballot_sync(kFull, value == top)) - 1;
      if (lane == owner) {
        some[at + (32 / kWarps) * warp + i] = top;
        value = 0;
      }
    }
  };
  next(0);
  if (wide) next(32);
}
// ... and then one warp finds the k-th, to some[0].
__device__ __forceinline__ void kth_largest(int k, bool wide, int lane, uint32_t* some) {
  const uint32_t v = some[lane], u = wide ? some[32 + lane] : 0u;
  int before = 0, before_u = wide ? 0 : 64;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint32_t w = __shfl_sync(kFull, v, i);
    before += w > v || (w == v && i < lane) ? 1 : 0;
  }
  if (wide) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t w = __shfl_sync(kFull, v, i), x = __shfl_sync(kFull, u, i);
      before += x > v ? 1 : 0;
      before_u += (w >= u ? 1 : 0) + (x > u || (x == u && i < lane) ? 1 : 0);
    }
  }
  __syncwarp();
  if (before == k - 1) some[0] = v;
  if (before_u == k - 1) some[0] = u;
}

// A CTA's share of a row's groups: blocks of kAhead, and what is left on either
// side (of a short share, all of it, so that every warp has some) one at a time; its
// warps take either in turn.
template <int kType, int kWarps>
struct Share {
  int g0, g1, inner0, blocks, tail;
  __device__ Share(const Row<kType>& row, int n, int rank, int split) {
    constexpr int kAhead = Logit<kType>::kAhead;
    g0 = (int)((long long)n * rank / split);
    g1 = (int)((long long)n * (rank + 1) / split);
    inner0 = row.shift > 0 ? max(g0, 1) : g0;
    const int inner = min(g1, (row.shift + row.V) / kGroup) - inner0;
    blocks = inner >= kWarps * kAhead ? inner / kAhead : 0;
    tail = inner0 + blocks * kAhead;
  }
  // the i-th of the single ones: groups [g0, inner0) and [tail, g1)
  __device__ int singles() const { return (inner0 - g0) + (g1 - tail); }
  __device__ int single(int i) const { return i < inner0 - g0 ? g0 + i : tail + i - (inner0 - g0); }
};

// One warp: the sum of lane `owner`'s logits in the groups of warp `warp` of a share,
// without the one that is `m`, the largest.
template <int kType, int kWarps>
__device__ __noinline__ float sum_beside(Row<kType> row, const Share<kType, kWarps> share, int warp, int lane,
                                        int owner, float m) {
  constexpr int kAhead = Logit<kType>::kAhead;
  const int in_blocks = (share.blocks - warp + kWarps - 1) / kWarps * kAhead;
  const int alone = (share.singles() - warp + kWarps - 1) / kWarps;
  float s = 0.0f;
  for (int i = lane; i < in_blocks + alone; i += 32) {
    const int g = i < in_blocks ? share.inner0 + (warp + i / kAhead * kWarps) * kAhead + i % kAhead
                                : share.single(warp + (i - in_blocks) * kWarps);
    float f[8];
    row.load_group(g, owner, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += f[j] == m ? 0.0f : exp2_approx(max_nan((f[j] - m) * kLog2e, kFarBelow));
  }
  return warp_sum(s);
}

// kWarps: 16, 8 or 4 warps a CTA, 32 an SM (64 registers a thread).
template <int kType, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps) logprobs_kernel(const LogprobParams p, int split) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Part s_warp[kWarps];
  __shared__ Part s_cta;
  __shared__ bool s_apart;
  __shared__ int s_sel[kMaxGroups];
  __shared__ uint32_t s_some[64];
  __shared__ int s_groups, s_count, s_few_count;
  __shared__ uint64_t s_cand[kMaxCandidates], s_few[kFewCandidates], s_round[2][kWarps];
  dev::griddep_launch_dependents();
  dev::griddep_wait();

  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int rank = split > 1 ? (int)dev::cluster_ctarank() : 0;
  const int row_index = (int)blockIdx.x / split;
  const Row<kType> row(p, row_index);
  const int n = row.groups();
  const Share<kType, kWarps> share(row, n, rank, split);
  uint32_t* s_best = reinterpret_cast<uint32_t*>(smem);              // [n] the groups' maxima

  Sums a{-INFINITY, 0.0f, 0.0f};
  float lane_top = -INFINITY;
  constexpr int kAhead = Logit<kType>::kAhead;
  // a warp's next block is loaded while it adds one
  const int inner0 = share.inner0, blocks = share.blocks;
  const auto load = [&](int block, uint4 (&w)[kAhead][Logit<kType>::kLoads]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) row.load_words(inner0 + block * kAhead + i, lane, w[i]);
  };
  uint4 next[kAhead][Logit<kType>::kLoads];
  if (warp < blocks) load(warp, next);
  for (int block = warp; block < blocks; block += kWarps) {
    uint4 w[kAhead][Logit<kType>::kLoads];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
#pragma unroll
      for (int q = 0; q < Logit<kType>::kLoads; ++q) w[i][q] = next[i][q];
    }
    if (block + kWarps < blocks) load(block + kWarps, next);
    float top = -INFINITY, mine = 0.0f;            // lane i writes down the block's group i's maximum
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float of_lane = Logit<kType>::max_of(w[i]), m = warp_max(of_lane);
      lane_top = fmaxf(lane_top, of_lane);
      mine = lane == i ? m : mine;
      top = fmaxf(top, m);
    }
    if (lane < kAhead) s_best[inner0 + block * kAhead + lane] = order_of(mine);
    if (top > a.m) a.rebase(top);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) add_words<kType>(a, w[i]);
  }
  for (int i = warp; i < share.singles(); i += kWarps) {
    const int g = share.single(i);
    float f[8];
    row.load_group(g, lane, f);
    float m = f[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, f[j]);
    lane_top = fmaxf(lane_top, m);
    m = warp_max(m);
    if (lane == 0) s_best[g] = order_of(m);
    if (m > a.m) a.rebase(m);
    add_any(a, f);
  }
  const int owner = (__ffs(__ballot_sync(kFull, lane_top == a.m)) - 1) & 31;
  const float rest = warp_sum(lane == owner ? 0.0f : a.s);
  a.s = warp_sum(a.s);
  a.t = warp_sum(a.t);
  if (lane == 0) s_warp[warp] = Part{a, rest, rank << 16 | warp << 8 | owner};
  if (threadIdx.x == 0) s_groups = s_count = 0;
  const bool some = p.k > 0;
  // k close to 32 would make the bound the least warp's (1024 x 131072 bf16, top 32:
  // 64 us, of 64 values 56; rows of few groups have few logits a lane to choose from:
  // 4096 x 1000 22.6 us, of 64 25.5; rows masked to some 20 logits pay 0.3-1.2 us for
  // it: 1 x 131072 7.6 and 8.8, 65 x 50001 f32 9.5 and 10.1)
  const bool wide = p.k > 24 && n > 24;
  if (some && split == 1) top_lanes<kWarps>(order_of(lane_top), wide, warp, lane, s_some);
  __syncthreads();
  // One warp joins the sums, and another looks for the bound meanwhile.
  constexpr int kJoins = kWarps - 1;
  const Part none{{-INFINITY, 0.0f, 0.0f}, 0.0f, 0};
  Part part = none;
  if (warp == kJoins && lane < kWarps) part = s_warp[lane];
  if (split > 1) {
    // the first CTA takes the others' sums and maxima from their shared memory
    if (warp == kJoins) {
      part = join(part);
      if (lane == 0) s_cta = part;
      __syncwarp();
    }
    dev::cluster_arrive_release();
    dev::cluster_wait_acquire();
    if (rank != 0) {
      dev::cluster_arrive_release();
      dev::cluster_wait_acquire();
      return;
    }
    if (warp == kJoins) {
      part = none;
      if (lane < split) {
        const uint32_t at = dev::mapa(dev::smem_u32(&s_cta), (uint32_t)lane);
        part = Part{{dev::ld_cluster_f32(at), dev::ld_cluster_f32(at + 4), dev::ld_cluster_f32(at + 8)},
                    dev::ld_cluster_f32(at + 12),
                    (int)dev::ld_cluster_u32(at + 16)};
      }
      __syncwarp();
    }
    if (some) {
      for (int g = share.g1 + (int)threadIdx.x; g < n; g += 32 * kWarps) {
        // the rank whose run of groups holds g
        const int r = (int)(((long long)(g + 1) * split - 1) / n);
        s_best[g] = dev::ld_cluster_u32(dev::mapa(dev::smem_u32(&s_best[g]), (uint32_t)r));
      }
      __syncthreads();
      // where other CTAs read a part of the row, the bound is of the groups' maxima
      uint32_t mine = 0;
      for (int g = n * warp / kWarps + lane; g < n * (warp + 1) / kWarps; g += 32) mine = max(mine, s_best[g]);
      top_lanes<kWarps>(mine, wide, warp, lane, s_some);
    }
    dev::cluster_arrive_release();
    __syncthreads();
  }
  if (warp == kJoins) {
    part = join(part);
    // The largest logit apart from the others where they add less than an eighth.
    const bool apart = part.sums.s < 1.125f && fabsf(part.sums.m) < INFINITY;
    if (apart) {
      part.sums.s = part.rest + sum_beside<kType, kWarps>(row, Share<kType, kWarps>(row, n, part.where >> 16, split),
                                                          part.where >> 8 & 255, lane, part.where & 255, part.sums.m);
    }
    if (lane == 0) s_cta = part, s_apart = apart;
  }
  if (some && warp == 0) kth_largest(p.k, wide, lane, s_some);
  __syncthreads();
  if (split > 1) dev::cluster_wait_acquire();
  const bool writes = (int)threadIdx.x == 32 * kJoins;       // the row's own results
  long long token = -1;
  if (writes && p.tokens != nullptr) token = p.tokens[row_index];

  int groups = 0, count = 0;
  const uint64_t* list = s_cand;
  if (some) {
    // The groups to read again: those whose maximum reaches the bound, and their
    // logits that do.  Where that is many (equal ones: a mask that leaves fewer
    // than k, say), those above the bound alone, and the row's first ones equal to
    // it; where even those groups are many, the k best groups.
    const uint32_t bound = s_some[0];
    const auto reaching = [&](uint32_t least_order) {
      for (int g = (int)threadIdx.x; g < n; g += 32 * kWarps) {
        if (s_best[g] >= least_order) {
          const int at = atomicAdd(&s_groups, 1);
          if (at < kMaxGroups) s_sel[at] = g;
        }
      }
      __syncthreads();
      return s_groups;
    };
    groups = reaching(bound);
    float least = value_of(bound);
    bool strict = false;
    const bool ordered = bound < order_of(INFINITY);         // a finite logit is above it, and it is no NaN
    // (a bound that is a mask's value is reached by every masked logit)
    for (bool again = groups > kMaxGroups || least <= Logit<kType>::kLowest;; again = true) {
      if (again) {
        __syncthreads();
        if (threadIdx.x == 0) s_groups = s_count = 0;
        __syncthreads();
        groups = reaching(bound + 1);
        strict = ordered && groups <= kMaxGroups;
        least = value_of(bound + 1);
        if (!strict) {
          groups = min(p.k, n);
          if (warp == 0) {
            const uint32_t last = draw_groups(s_best, n, groups, lane, s_sel);
            if (lane == 0) s_some[0] = last;
          }
          __syncthreads();
          least = value_of(s_some[0]);
        }
      }
      for (int i = warp; i < groups; i += kWarps) {
        const int g = s_sel[i];
        float f[8];
        row.load_group(g, lane, f);
        uint32_t in = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) in |= f[j] < least ? 0u : 1u << j;
        // a lane has hardly ever more than one, which is read again by its place
        for (; in != 0; in &= in - 1) {
          const int id = Row<kType>::at(g, lane, __ffs(in) - 1) - row.shift;
          if (id < 0 || id >= p.V) continue;
          const int at = atomicAdd(&s_count, 1);
          if (at < kMaxCandidates) s_cand[at] = key_of(order_of(Logit<kType>::one(row.x[id])), id);
        }
      }
      __syncthreads();
      count = s_count;
      if (count > kFewCandidates && count <= kMaxCandidates) {
        // The same again for the list (a short row's lanes have few logits, so its
        // bound is low): its parts' largest give a closer bound.
        uint32_t top = 0;
        for (int c = kWarps * lane + warp; c < count; c += 32 * kWarps) top = max(top, (uint32_t)(s_cand[c] >> 32));
        top_lanes<kWarps>(top, wide, warp, lane, s_some);
        __syncthreads();
        if (warp == 0) kth_largest(p.k, wide, lane, s_some);
        if (threadIdx.x == 32) s_few_count = 0;
        __syncthreads();
        const uint32_t closer = s_some[0];
        for (int c = (int)threadIdx.x; c < count; c += 32 * kWarps) {
          const uint64_t key = s_cand[c];
          if ((uint32_t)(key >> 32) >= closer) {
            const int at = atomicAdd(&s_few_count, 1);
            if (at < kFewCandidates) s_few[at] = key;
          }
        }
        __syncthreads();
        if (s_few_count <= kFewCandidates) count = s_few_count, list = s_few;
      }
      if (again || count <= kFewCandidates || !ordered) break;
    }
    if (strict && count < p.k) {
      if (warp == 0) first_equal<kType>(row, s_best, n, bound, value_of(bound), lane, p.k - count, s_cand + count);
      count = p.k;
      __syncthreads();
    }
  }

  const Sums all = s_cta.sums;
  const float total = s_apart ? 1.0f + all.s : all.s;
  // a row whose every logit is masked: no probabilities (log 0), entropy 0
  const float log_s = s_apart ? log1pf(all.s) : total == 0.0f ? 0.0f : logf(total);
  const float base = all.m == -INFINITY && total == 0.0f ? 0.0f : all.m;
  if (writes) {
    p.entropy[row_index] = total == 0.0f ? 0.0f : log_s - kLn2 * (all.t / total);
    if (p.tokens != nullptr) {
      p.logprob[row_index] = token >= 0 && token < (long long)p.V ? (Logit<kType>::one(row.x[token]) - base) - log_s
                                                                  : __uint_as_float(0x7FC00000u);
    }
  }
  if (!some) return;

  // Their order is by (logit, lowest index), each one's place in it the
  // number before it, so how they came into the list does not matter.
  long long* ids = p.top_ids + (long long)row_index * p.k;
  float* tops = p.top_logprobs + (long long)row_index * p.k;
  if (count <= kFewCandidates) {
    // four lanes count for one
    for (int c0 = 8 * warp; c0 < count; c0 += 8 * kWarps) {
      const int c = c0 + (lane >> 2);
      const uint64_t key = list[min(c, count - 1)];
      int before = 0;
      for (int i = lane & 3; i < count; i += 4) before += list[i] > key ? 1 : 0;
      before += __shfl_xor_sync(kFull, before, 1);
      before += __shfl_xor_sync(kFull, before, 2);
      if ((lane & 3) == 0 && c < count && before < p.k) {
        ids[before] = id_of(key);
        tops[before] = (value_of((uint32_t)(key >> 32)) - base) - log_s;
      }
    }
    return;
  }
  // More (a short row, a sorted one, many equal logits): one alternative after
  // another, from the list, or where that did not hold them from the groups again.
  uint64_t last = ~0ull;
  for (int r = 0; r < p.k; ++r) {
    uint64_t best = 0;
    if (count <= kMaxCandidates) {
      for (int c = (int)threadIdx.x; c < count; c += 32 * kWarps) {
        const uint64_t key = s_cand[c];
        if (key < last && key > best) best = key;
      }
    } else {
      for (int i = warp; i < groups; i += kWarps) {
        float f[8];
        row.load_group(s_sel[i], lane, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int id = Row<kType>::at(s_sel[i], lane, j) - row.shift;
          const uint64_t key = key_of(order_of(f[j]), id);
          if (id >= 0 && id < p.V && key < last && key > best) best = key;
        }
      }
    }
    best = warp_max64(best);
    if (lane == 0) s_round[r & 1][warp] = best;
    __syncthreads();
    last = s_round[r & 1][0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) last = s_round[r & 1][i] > last ? s_round[r & 1][i] : last;
    if (threadIdx.x == 0) {
      ids[r] = id_of(last);
      tops[r] = (value_of((uint32_t)(last >> 32)) - base) - log_s;
    }
  }
}

// Shared memory: the groups' maxima (one more group than the row fills when
// it starts inside a word).
size_t logprob_smem(int V) { return ((size_t)V + 7u + kGroup - 1u) / kGroup * 4u; }

template <int kType, int kWarps>
cudaError_t launch_warps(const LogprobParams& p, int split, cudaStream_t stream) {
  return launch_chained(logprobs_kernel<kType, kWarps>, dim3((unsigned)p.rows * (unsigned)split), dim3(32 * kWarps),
                        logprob_smem(p.V), (unsigned)split, stream, p, split);
}

template <int kType>
cudaError_t launch_logprobs(const LogprobParams& p, int split, int warps, cudaStream_t stream) {
  return warps == 4   ? launch_warps<kType, 4>(p, split, stream)
         : warps == 8 ? launch_warps<kType, 8>(p, split, stream)
                      : launch_warps<kType, 16>(p, split, stream);
}

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

}  // namespace

cudaError_t prepare_logprobs(int (&clusters)[3]) {
  const int most = (int)logprob_smem(kMaxVocab);
  cudaError_t e = cudaSuccess;
  const auto set = [&](auto* kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  };
  set(logprobs_kernel<1, 4>), set(logprobs_kernel<2, 4>), set(logprobs_kernel<3, 4>);
  set(logprobs_kernel<1, 8>), set(logprobs_kernel<2, 8>), set(logprobs_kernel<3, 8>);
  set(logprobs_kernel<1, 16>), set(logprobs_kernel<2, 16>), set(logprobs_kernel<3, 16>);
  for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2u << i;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2u << i);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = (size_t)most;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters[i], logprobs_kernel<2, 16>, &cfg);
  }
  return e;
}

}  // namespace splitk

using namespace splitk;

extern "C" {

SPLITK_API int splitk_logprobs(const void* logits, int logits_type, long long stride, const long long* tokens,
                               float* logprob, float* entropy, int top_k, long long* top_ids, float* top_logprobs,
                               int M, int V, splitk_stream_t stream) {
  if (!logits || !entropy || (tokens != nullptr) != (logprob != nullptr)) return SPLITK_ERR_NULL;
  if (top_k > 0 && (!top_ids || !top_logprobs)) return SPLITK_ERR_NULL;
  if (logits_type != SPLITK_DTYPE_BF16 && logits_type != SPLITK_DTYPE_F32 && logits_type != SPLITK_DTYPE_F16) {
    return SPLITK_ERR_INVALID_ARGUMENT;
  }
  if (M < 1 || V < 1 || V > kMaxVocab || stride < V || M > (1 << 27)) return SPLITK_ERR_INVALID_SHAPE;
  if (top_k < 0 || top_k > kMaxTop || top_k > V) return SPLITK_ERR_INVALID_ARGUMENT;
  if (!aligned(logits, logits_type == SPLITK_DTYPE_F32 ? 4u : 2u) || !aligned(tokens, 8) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || (top_k > 0 && (!aligned(top_ids, 8) || !aligned(top_logprobs, 4)))) {
    return SPLITK_ERR_MISALIGNED;
  }
  DeviceSize dev;
  int rc = require_logprobs(&dev);
  if (rc != SPLITK_OK) return rc;
  const LogprobParams p{logits, stride, tokens, logprob, entropy, top_ids, top_logprobs, M, V, top_k};
  // CTAs sharing a row of 128 KB or more (shorter ones gain less than a cluster
  // costs: bf16, top 20, 30 x 32000 6.2 us in one CTA and 7.3 in eight, 30 x 131072
  // 9.9 in two and 8.7 in eight): as many as leave each row's cluster a place at
  // once (38 x 131072: 10.1 us in four, 12.7 in eight, which do not all fit).
  int split = 1;
  if ((long long)V * (logits_type == SPLITK_DTYPE_F32 ? 4 : 2) >= 1ll << 17) {
    for (int i = 0; i < 3 && M <= dev.row_clusters[i]; ++i) split = 2 << i;
  }
  // Few rows get large CTAs, for their latency.  Rows enough to fill the device
  // get smaller ones, so that more rows are at their different stages at once, the
  // more so the less there is to a row (bf16, top 20, with 4, 8 and 16 warps: 100 x
  // 8000 6.5, 5.7 and 5.7 us; 400 x 16000 11.4, 10.4, 13.8; 1024 x 8000 12.7, 15.3,
  // 21.0; 1024 x 65536 36, 31, 36; 4096 x 32000 65, 71, 101; 400 x 131072 39, 31, 25;
  // 1024 x 131072 61, 52, 55).  A warp has a group at least, or a row's bound is
  // of too few lanes.
  int warps = split > 1 || 2ll * M <= 3ll * dev.num_sms ? 16
              : V > 65536                               ? (M < 4 * dev.num_sms ? 16 : 8)
                                                        : (M < (V <= 16384 ? 4 : 12) * dev.num_sms ? 8 : 4);
  while (warps > 4 && V + kGroup / 2 < warps * kGroup) warps /= 2;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_type == SPLITK_DTYPE_BF16  ? launch_logprobs<1>(p, split, warps, s)
                        : logits_type == SPLITK_DTYPE_F32 ? launch_logprobs<2>(p, split, warps, s)
                                                          : launch_logprobs<3>(p, split, warps, s);
  return launched(e);
}

}  // extern "C"
