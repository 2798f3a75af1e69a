// splitk_adjust_logits(): penalties for repeated tokens, biases and grammar masks on
// a vocabulary's logits, in one pass over them.
//
// For a logit x of row m (f32), with `said` whether its token is in the row's
// history and `count` how often it is there behind the prompt:
//
//   said:       x = x > 0 ? x / repetition : x * repetition
//   count > 0:  x = x - frequency * count;  x = x - presence
//   biased:     x = x + bias
//   banned:     x = -inf
//
// each an f32 operation of its own, rounded once more to the logits' type.
//
// A CTA takes a span of a row's vocabulary.  Its threads pass the logits on as they are
// (banned ones as -inf, which need not be read), while they count those of the row's
// history that lie in the span in shared memory (whole numbers: any order gives the
// same) and list the tokens that they meet; then they go over the listed tokens one by
// one.  Memory is the bound: each logit is read and written once, the history read
// once for each span, from L2: 256 x 131072 bf16 logits take 22.6 us (5.9 TB/s), 46 with
// histories of 4096, 64 biases and masks (a span's three dependent phases, with two CTAs
// an SM beside each other); one row of 131072 3.3 us.  (Looking at every logit's count on its way took 224
// instructions for eight of each of a warp's lanes, since some lane always has a
// counted one: 256 x 131072 logits with histories of 4096 tokens 51-86 us.)

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "splitk.h"
#include "splitk_device.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

constexpr int kMaxBias = 1024;

struct AdjustParams {
  const void* logits;
  long long stride, out_stride;
  void* out;
  splitk_adjust_t how;
  int V, spans;             // CTAs of a row
  bool in_place;
};

// An element's bits as f32 and back (kType: SPLITK_DTYPE_*).
template <int kType>
__device__ __forceinline__ float value_of(uint32_t bits) {
  if (kType == SPLITK_DTYPE_F32) return __uint_as_float(bits);
  if (kType == SPLITK_DTYPE_BF16) return __uint_as_float(bits << 16);
  float f;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(bits));
  return f;
}
template <int kType>
__device__ __forceinline__ uint32_t bits_of(float v) {
  if (kType == SPLITK_DTYPE_F32) return __float_as_uint(v);
  uint32_t r;
  if (kType == SPLITK_DTYPE_BF16) return dev::pack_bf16x2(v, 0.0f) & 0xFFFFu;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFFFu;
}
// What a banned logit becomes.
template <int kType>
__device__ __forceinline__ constexpr uint32_t minus_infinity() {
  return kType == SPLITK_DTYPE_F32 ? 0xFF800000u : kType == SPLITK_DTYPE_BF16 ? 0xFF80u : 0xFC00u;
}

// A token's word: 2 for each time behind the prompt, 1 more (once) for one of the
// prompt, kBiased for one that has a bias, kTwice for one that has several.
constexpr uint32_t kBiased = 0x80000000u, kTwice = 0x40000000u;
constexpr int kMaxHistory = 1 << 28;       // counts stay below

// A row's biases: the slot of each in the span, or kOutside, and its value, by place in
// the row's list; and the places of those that lie in the span, in any order.
constexpr uint32_t kOutside = 0xFFFFu;
struct BiasList {
  int count;                               // that lie in the span
  uint16_t place[kMaxBias];
  alignas(16) uint16_t slot[kMaxBias];     // to a multiple of eight
  alignas(16) float value[kMaxBias];       // of those that lie in the span
};

// The sum of a slot's biases in the list's order, for its first one alone (at `place`):
// false for the others.  One pass over the list's `n` slots, eight a load: whether any of
// two is the one looked for is whether their difference has a zero half.  The eight
// values are there before the first is needed, and nothing branches between additions.
// (1 x 131072 bf16, 1024 biases of one token 29 us, of 512 tokens twice 39, of
// different ones 4.3; with a pass of the list for each addition 98600 and 427.)
__device__ __noinline__ bool bias_sum(const BiasList& list, int n, int place, float* sum) {
  const uint32_t slot = list.slot[place], both = slot * 0x10001u;
  const uint4* eights = reinterpret_cast<const uint4*>(list.slot);
  float total = list.value[place];
#pragma unroll 2
  for (int first = 0; first < n; first += 8) {
    const uint4 q = eights[first / 8];
    const uint32_t w[4] = {q.x ^ both, q.y ^ both, q.z ^ both, q.w ^ both};
    uint32_t zero = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) zero |= (w[i] - 0x00010001u) & ~w[i] & 0x80008000u;
    if (zero == 0u) continue;
    if (first + 8 <= place) return false;
    const float4 lo = *reinterpret_cast<const float4*>(list.value + first), hi = *reinterpret_cast<const float4*>(list.value + first + 4);
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool hit = (w[i / 2] & (i % 2 ? 0xFFFF0000u : 0xFFFFu)) == 0u;
      if (hit && first + i < place) return false;
      const float next = __fadd_rn(total, v[i]);
      total = hit && first + i > place ? next : total;
    }
  }
  *sum = total;
  return true;
}

// A row's numbers.
struct RowNumbers {
  float repetition, presence, frequency;
  int length, prompt;
  __device__ __forceinline__ RowNumbers(const splitk_adjust_t& h, int row) {
    repetition = h.repetition ? h.repetition[row] : 1.0f;
    presence = h.presence ? h.presence[row] : 0.0f;
    frequency = h.frequency ? h.frequency[row] : 0.0f;
    const long long most = h.history_length;
    length = (int)(h.lengths ? max(0ll, min(h.lengths[row], most)) : most);
    prompt = h.prompt_lengths ? (int)max(0ll, min(h.prompt_lengths[row], most)) : 0;
  }
  __device__ __forceinline__ float apply(float x, uint32_t word) const {
    const uint32_t said = word & ~(kBiased | kTwice), count = said >> 1;
    if (said != 0u) x = x > 0.0f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
    if (count != 0u) x = __fsub_rn(__fsub_rn(x, __fmul_rn(frequency, (float)count)), presence);
    return x;
  }
};

template <int kType>
constexpr int kSize = kType == SPLITK_DTYPE_F32 ? 4 : 2;
template <int kType>
__device__ __forceinline__ uint32_t load_one(const void* p, long long at) {
  return kType == SPLITK_DTYPE_F32 ? static_cast<const uint32_t*>(p)[at] : (uint32_t)static_cast<const uint16_t*>(p)[at];
}
template <int kType>
__device__ __forceinline__ void store_one(void* p, long long at, uint32_t bits) {
  if (kType == SPLITK_DTYPE_F32) {
    static_cast<uint32_t*>(p)[at] = bits;
  } else {
    static_cast<uint16_t*>(p)[at] = (uint16_t)bits;
  }
}

// kEach bits of a row's `allowed` from logit e on, all of them the row's.
template <int kEach>
__device__ __forceinline__ uint32_t allowed_bits(const uint32_t* words, int e) {
  constexpr uint32_t kAll = (1u << kEach) - 1u;
  const int at = e >> 5, shift = e & 31;
  if (e % 8 == 0) return reinterpret_cast<const uint8_t*>(words)[e / 8] & kAll;
  uint32_t v = words[at] >> shift;
  if (shift > 32 - kEach) v |= words[at + 1] << (32 - shift);
  return v & kAll;
}

// 16 bytes of logits with those that have no bit in `keep` banned.
template <int kType>
__device__ __forceinline__ uint4 ban(uint4 v, uint32_t keep) {
  constexpr uint32_t kInf = minus_infinity<kType>();
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kType == SPLITK_DTYPE_F32) {
      w[i] = (keep >> i) & 1u ? w[i] : kInf;
    } else {
      const uint32_t two = keep >> (2 * i), mask = ((two & 1u) | ((two & 2u) << 15)) * 0xFFFFu;
      w[i] = (w[i] & mask) | (kInf * 0x10001u & ~mask);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 16 bytes from `shift` bytes (a logit's size times any number, below 16) behind
// the start of `v` on, `u` being the next 16.
__device__ __forceinline__ uint4 shifted(uint4 v, uint4 u, int shift) {
  const uint32_t w[8] = {v.x, v.y, v.z, v.w, u.x, u.y, u.z, u.w};
  const uint32_t bits = 8u * ((uint32_t)shift & 3u);
  uint32_t o[4];
  const auto from = [&](auto first) {
    constexpr int k = decltype(first)::value;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[k + i], w[k + i + 1 < 8 ? k + i + 1 : 7], bits);
  };
  switch (shift >> 2) {                    // the same for all threads of a CTA
    case 0: from(std::integral_constant<int, 0>{}); break;
    case 1: from(std::integral_constant<int, 1>{}); break;
    case 2: from(std::integral_constant<int, 2>{}); break;
    default: from(std::integral_constant<int, 3>{}); break;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Threads resident an SM: 40 registers each for CTAs that are many and read short
// histories, else 64.
__host__ __device__ constexpr int threads_an_sm(int threads, int vecs) { return threads == 256 && vecs == 4 ? 1536 : 1024; }

// kVecs times 16 bytes of a row of `out` a thread, from the 16-byte boundary before
// the row's start on.  Where the row of logits lies otherwise between boundaries, a
// vector is cut out of the two around it.  What a row's ends leave of a vector, or
// would have read outside the row, goes a logit at a time.
template <int kType, int kThreads, int kVecs>
__global__ void __launch_bounds__(kThreads, threads_an_sm(kThreads, kVecs) / kThreads) adjust_kernel(const AdjustParams p) {
  constexpr int kEach = 16 / kSize<kType>, kSpan = kThreads * kEach * kVecs;
  static_assert(kSpan <= kOutside, "a slot has 16 bits");
  extern __shared__ uint4 s_words[];                    // [kSpan] words, then the tokens met
  uint32_t* words = reinterpret_cast<uint32_t*>(s_words);
  uint16_t* met = reinterpret_cast<uint16_t*>(words + kSpan);
  __shared__ BiasList list;
  __shared__ int met_count;
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const splitk_adjust_t& h = p.how;
  const int row = (int)(blockIdx.x / (unsigned)p.spans), tid = (int)threadIdx.x;
  const uint8_t* logits = static_cast<const uint8_t*>(p.logits) + (long long)row * p.stride * kSize<kType>;
  uint8_t* out = static_cast<uint8_t*>(p.out) + (long long)row * p.out_stride * kSize<kType>;
  const int past = (int)((uintptr_t)out % 16) / kSize<kType>;
  const int lo = (int)(blockIdx.x % (unsigned)p.spans) * kSpan - past;
  const bool marked = h.history_length > 0 || h.bias_count > 0;
  const uint32_t* allowed =
      h.allowed ? reinterpret_cast<const uint32_t*>(h.allowed) + (long long)row * ((p.V + 31) / 32) : nullptr;

  // the first tokens of the history, without waiting for its length
  constexpr int kTokens = threads_an_sm(kThreads, kVecs) > 1024 ? 4 : 8;        // a thread's loads at once
  long long id[kTokens];
  const auto load_tokens = [&](long long first, int end) {
    const long long* tokens = h.history + (long long)row * h.history_length;
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const long long i = first + j * kThreads;
      id[j] = i < end ? tokens[i] : -1;
    }
  };
  const RowNumbers numbers(h, row);
  const long long* bias_ids = h.bias_ids + (long long)row * h.bias_count;
  const float* biases = h.bias_values + (long long)row * h.bias_count;
  long long bias_id = tid < h.bias_count ? bias_ids[tid] : -1;
  float bias = tid < h.bias_count ? biases[tid] : 0.0f;
  if (kVecs < 4) load_tokens(tid, h.history_length);
  if (marked) {
#pragma unroll
    for (int i = 0; i < kSpan / 4 / kThreads; ++i) s_words[i * kThreads + tid] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) list.count = 0, met_count = 0;
  }

  // ---- the logits as they are
  constexpr uint32_t kAll = (1u << kEach) - 1u;
  // bytes between the boundary before a vector's logits and their start
  const int shift = (int)(((uintptr_t)logits - (uintptr_t)past * kSize<kType>) % 16), margin = shift != 0 ? kEach : 0;
  uint32_t keep[kVecs];                                 // of the vectors that are the row's with what is read around them
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int e = lo + (i * kThreads + tid) * kEach;
    keep[i] = e < margin || e + kEach + margin > p.V ? ~0u : allowed ? allowed_bits<kEach>(allowed, e) : kAll;
  }
  const uint8_t* from = logits + (long long)(lo + tid * kEach) * kSize<kType> - shift;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (keep[i] != 0u && keep[i] != ~0u && !(p.in_place && keep[i] == kAll)) {
      v[i] = *reinterpret_cast<const uint4*>(from + i * kThreads * 16);
    }
  }
  if (kVecs >= 4) load_tokens(tid, numbers.length);
  uint8_t* into = out + (long long)(lo + tid * kEach) * kSize<kType>;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (keep[i] == ~0u) {
      const int e = lo + (i * kThreads + tid) * kEach;
#pragma unroll 1
      for (int j = max(e, 0); j < min(e + kEach, p.V); ++j) {
        const bool kept = !allowed || ((allowed[j >> 5] >> (j & 31)) & 1u) != 0u;
        if (!(kept && p.in_place)) store_one<kType>(out, j, kept ? load_one<kType>(logits, j) : minus_infinity<kType>());
      }
      continue;
    }
    if (p.in_place && keep[i] == kAll) continue;
    if (shift != 0 && keep[i] != 0u) {
      v[i] = shifted(v[i], *reinterpret_cast<const uint4*>(from + i * kThreads * 16 + 16), shift);
    }
    if (keep[i] != kAll) v[i] = ban<kType>(v[i], keep[i]);
    *reinterpret_cast<uint4*>(into + i * kThreads * 16) = v[i];
  }
  if (!marked) return;

  // ---- the span's tokens counted
  __syncthreads();
  for (long long first = tid;;) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const uint32_t at = (uint32_t)id[j] - (uint32_t)lo;
      const long long i = first + j * kThreads;
      if ((unsigned long long)id[j] >= (unsigned long long)p.V || at >= (uint32_t)kSpan || i >= numbers.length) continue;
      const uint32_t before = i >= numbers.prompt ? atomicAdd(&words[at], 2u) : atomicOr(&words[at], 1u);
      if (before == 0u) met[atomicAdd(&met_count, 1)] = (uint16_t)at;
    }
    first += kTokens * kThreads;
    if (first - tid >= numbers.length) break;
    load_tokens(first, numbers.length);
  }
  for (int b = tid; b < ((h.bias_count + 7) & ~7); b += kThreads) {
    if (b != tid) bias_id = b < h.bias_count ? bias_ids[b] : -1, bias = b < h.bias_count ? biases[b] : 0.0f;
    const uint32_t at = (uint32_t)bias_id - (uint32_t)lo;
    const bool in = (unsigned long long)bias_id < (unsigned long long)p.V && at < (uint32_t)kSpan;
    list.slot[b] = (uint16_t)(in ? at : kOutside);
    if (!in) continue;
    if ((atomicOr(&words[at], kBiased) & kBiased) != 0u) atomicOr(&words[at], kTwice);
    list.place[atomicAdd(&list.count, 1)] = (uint16_t)b, list.value[b] = bias;
  }
  __syncthreads();

  // ---- and changed, over what another thread has stored: those that were met and
  // have no bias, and those that have
  for (int i = tid; i < met_count + list.count; i += kThreads) {
    const int b = i < met_count ? -1 : list.place[i - met_count];
    const uint32_t at = b < 0 ? met[i] : list.slot[b], word = words[at];
    const int e = lo + (int)at;
    const uint32_t bits = load_one<kType>(logits, e);
    const uint32_t ok = allowed ? allowed[e >> 5] >> (e & 31) : 1u;
    float sum = 0.0f;
    if (b < 0) {
      if ((word & kBiased) != 0u) continue;
    } else if ((word & kTwice) == 0u) {
      sum = list.value[b];
    } else if (!bias_sum(list, h.bias_count, b, &sum)) {
      continue;
    }
    if ((ok & 1u) == 0u) continue;
    float x = numbers.apply(value_of<kType>(bits), word);
    if (b >= 0) x = __fadd_rn(x, sum);
    store_one<kType>(out, e, bits_of<kType>(x));
  }
}

// A kernel's shared memory: words of the span, and as many of its tokens as are met.
template <int kType, int kThreads, int kVecs>
constexpr int kSpanOf = kThreads * (16 / kSize<kType>) * kVecs;
constexpr size_t smem_of(int span, int met) { return (size_t)span * 4 + (size_t)met * 2; }

template <int kType, int kThreads, int kVecs>
cudaError_t launch_adjust(AdjustParams& p, int M, cudaStream_t stream) {
  constexpr int kEach = 16 / kSize<kType>, kSpan = kSpanOf<kType, kThreads, kVecs>;
  // (a row's start may be past a boundary: all of them alike, or by any number of logits)
  const int past = p.out_stride % kEach == 0 ? (int)((uintptr_t)p.out % 16) / kSize<kType> : kEach - 1;
  p.spans = (p.V + past + kSpan - 1) / kSpan;
  const bool marked = p.how.history_length > 0 || p.how.bias_count > 0;
  return launch_chained(adjust_kernel<kType, kThreads, kVecs>, dim3((unsigned)((long long)M * p.spans)), dim3(kThreads),
                        marked ? smem_of(kSpan, std::min(kSpan, p.how.history_length)) : 0, 1, stream, p);
}

template <int kType, int kThreads, int kVecs>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(adjust_kernel<kType, kThreads, kVecs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_of(kSpanOf<kType, kThreads, kVecs>, kSpanOf<kType, kThreads, kVecs>));
}

// Long spans read the history fewer times and have more loads in flight; short ones
// fill the SMs and are the shortest chains of latencies.  Measured (us) with 256 x 1
// vectors, 512 x 2, 256 x 4 and 512 x 4 a CTA: 1 x 131072 bf16, 1500 tokens 3.4, 3.5,
// 4.8, 4.2; 64 x 32000 bf16, 1000 tokens 7.5, 5.1, 7.2, 6.4; 65 x 50001 f32, 300 tokens
// 15.9, 13.3, 8.5, 12.2; 256 x 131072 bf16, 4096 tokens 113, 66, 60, 46, without 39, 29,
// 22.3, 22.6; 256 x 50001 bf16, 1000 tokens 32, 23, 19.2, 18.2.
template <int kType>
cudaError_t choose_adjust(AdjustParams& p, int M, const DeviceSize& dev, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};                // a bit a device
  static_assert(kMaxDevices <= 64, "");
  const uint64_t bit = 1ull << dev.device;
  if ((ready.load() & bit) == 0) {
    cudaError_t e = allow_smem<kType, 256, 1>();
    if (e == cudaSuccess) e = allow_smem<kType, 512, 2>();
    if (e == cudaSuccess) e = allow_smem<kType, 256, 4>();
    if (e == cudaSuccess) e = allow_smem<kType, 512, 4>();
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  constexpr int kEach = 16 / kSize<kType>;
  const long long vectors = (long long)M * ((p.V + kEach - 1) / kEach);
  if (vectors <= (long long)dev.num_sms * 1024) return launch_adjust<kType, 256, 1>(p, M, stream);
  if (vectors <= (long long)dev.num_sms * 2048) return launch_adjust<kType, 512, 2>(p, M, stream);
  return p.how.history_length > 512 ? launch_adjust<kType, 512, 4>(p, M, stream) : launch_adjust<kType, 256, 4>(p, M, stream);
}

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

}  // namespace

}  // namespace splitk

using namespace splitk;

extern "C" {

SPLITK_API int splitk_adjust_logits(const void* logits, int type, long long stride, const splitk_adjust_t* how, void* out,
                                    long long out_stride, int M, int V, splitk_stream_t stream) {
  if (!logits || !out || !how) return SPLITK_ERR_NULL;
  const splitk_adjust_t& h = *how;
  if (type != SPLITK_DTYPE_BF16 && type != SPLITK_DTYPE_F32 && type != SPLITK_DTYPE_F16) return SPLITK_ERR_INVALID_ARGUMENT;
  if (M < 1 || V < 1 || V > (1 << 22) || stride < V || out_stride < V) return SPLITK_ERR_INVALID_SHAPE;
  if (h.history_length < 0 || h.history_length > kMaxHistory || h.bias_count < 0 || h.bias_count > kMaxBias) {
    return SPLITK_ERR_INVALID_ARGUMENT;
  }
  if ((h.history_length > 0 && !h.history) || (h.bias_count > 0 && (!h.bias_ids || !h.bias_values))) return SPLITK_ERR_NULL;
  if (!h.history && (h.lengths || h.prompt_lengths || h.repetition || h.presence || h.frequency)) return SPLITK_ERR_NULL;
  const uintptr_t size = type == SPLITK_DTYPE_F32 ? 4u : 2u;
  if (!aligned(logits, size) || !aligned(out, size) || !aligned(h.history, 8) || !aligned(h.lengths, 8) ||
      !aligned(h.prompt_lengths, 8) || !aligned(h.repetition, 4) || !aligned(h.presence, 4) || !aligned(h.frequency, 4) ||
      !aligned(h.bias_ids, 8) || !aligned(h.bias_values, 4) || !aligned(h.allowed, 4)) {
    return SPLITK_ERR_MISALIGNED;
  }
  if (out == logits && M > 1 && stride != out_stride) return SPLITK_ERR_INVALID_ARGUMENT;    // rows over other rows
  // a launch's CTAs, of at least 1024 logits
  if ((long long)M * (V / 1024 + 2) > 0x7FFFFFFFll) return SPLITK_ERR_INVALID_SHAPE;
  DeviceSize dev;
  const int rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  AdjustParams p{logits, stride, out_stride, out, h, V, 1, out == logits};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = type == SPLITK_DTYPE_F32   ? choose_adjust<SPLITK_DTYPE_F32>(p, M, dev, s)
                        : type == SPLITK_DTYPE_F16 ? choose_adjust<SPLITK_DTYPE_F16>(p, M, dev, s)
                                                   : choose_adjust<SPLITK_DTYPE_BF16>(p, M, dev, s);
  return launched(e);
}

}  // extern "C"
