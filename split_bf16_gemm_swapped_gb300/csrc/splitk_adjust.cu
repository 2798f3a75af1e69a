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
// A CTA takes a span of one row's vocabulary.  It counts those of the row's history
// that lie in the span in shared memory (whole numbers: any order gives the same),
// while the span's logits are on their way to its threads' registers; a word of zero
// says that a logit stays as it is.  Memory is the bound: each logit is read (but for
// eight banned ones in a row, and in place for all that do not change) and written
// once; the history is read once for each span, from L2.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
  int V, spans;
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
// prompt, kBiased for one that has a bias.
constexpr uint32_t kBiased = 0x80000000u;

// A row's biases that lie in the span: slot and place in the list, in any order.
struct BiasList {
  int count;
  uint32_t entry[kMaxBias];                // place << 16 | slot
};

// How a row's tokens change.
struct Changes {
  float repetition, presence, frequency;
  const float* bias;
  __device__ __forceinline__ Changes(const splitk_adjust_t& h, int row)
      : repetition(h.repetition ? h.repetition[row] : 1.0f), presence(h.presence ? h.presence[row] : 0.0f),
        frequency(h.frequency ? h.frequency[row] : 0.0f), bias(h.bias_values + (long long)row * h.bias_count) {}
  // The sum of a slot's biases in the list's order.
  __device__ __noinline__ float sum(const BiasList& list, uint32_t slot) const {
    float total = 0.0f;
    for (int last = -1, found = 0;; ++found) {
      int next = kMaxBias;                 // the place after `last`
      for (int i = 0; i < list.count; ++i) {
        const int place = (int)(list.entry[i] >> 16);
        if ((list.entry[i] & 0xFFFFu) == slot && place > last) next = min(next, place);
      }
      if (next == kMaxBias) return total;
      total = found == 0 ? bias[next] : __fadd_rn(total, bias[next]);
      last = next;
    }
  }
  __device__ __forceinline__ float apply(float x, uint32_t word, const BiasList& list, uint32_t slot) const {
    const uint32_t said = word & ~kBiased, count = said >> 1;
    if (said != 0u) x = x > 0.0f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
    if (count != 0u) x = __fsub_rn(__fsub_rn(x, __fmul_rn(frequency, (float)count)), presence);
    return (word & kBiased) != 0u ? __fadd_rn(x, sum(list, slot)) : x;
  }
};

// The words of the span [lo, lo + kSpan) and its biases; the caller's threads have
// passed a barrier when it returns.
template <int kThreads, int kSpan>
__device__ __forceinline__ void mark(const splitk_adjust_t& h, int row, int lo, int V, uint32_t* words, BiasList& list) {
  const int tid = (int)threadIdx.x;
  for (int i = tid; i < kSpan / 4; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) list.count = 0;
  __syncthreads();
  // a token's slot, kSpan or more outside the span or the vocabulary
  const auto slot_of = [&](long long id) { return (unsigned long long)id < (unsigned long long)V ? (uint32_t)((int)id - lo) : ~0u; };
  if (h.history_length > 0) {
    const int most = h.history_length;
    const int n = h.lengths ? (int)max(0ll, min(h.lengths[row], (long long)most)) : most;
    const long long prompt = h.prompt_lengths ? h.prompt_lengths[row] : 0;
    const long long* tokens = h.history + (long long)row * most;
    constexpr int kAtOnce = 8;             // loads in flight a thread
    for (int first = tid; first < n; first += kAtOnce * kThreads) {
      long long id[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const long long i = (long long)first + j * kThreads;
        id[j] = i < n ? tokens[i] : -1;
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const uint32_t at = slot_of(id[j]);
        if (at >= (uint32_t)kSpan) continue;
        if ((long long)first + j * kThreads >= prompt) {
          atomicAdd(&words[at], 2u);
        } else {
          atomicOr(&words[at], 1u);
        }
      }
    }
  }
  for (int b = tid; b < h.bias_count; b += kThreads) {
    const uint32_t at = slot_of(h.bias_ids[(long long)row * h.bias_count + b]);
    if (at >= (uint32_t)kSpan) continue;
    atomicOr(&words[at], kBiased);
    list.entry[atomicAdd(&list.count, 1)] = ((uint32_t)b << 16) | at;
  }
  __syncthreads();
}

// The eight bits of a row's `allowed` from logit e on (e > -8, < V).
__device__ __forceinline__ uint32_t allowed_bits(const uint32_t* words, int e, int V) {
  if (e < 0) return (words[0] << -e) & 0xFFu;
  const int at = e >> 5, shift = e & 31;
  uint32_t v = words[at] >> shift;
  if (shift > 24 && 32 * (at + 1) < V) v |= words[at + 1] << (32 - shift);
  return v & 0xFFu;
}

// Eight logits' bits: packed words in the 16-bit types.
template <int kType>
struct Group {
  static constexpr bool kHalf = kType != SPLITK_DTYPE_F32;
  static constexpr int kWords = kHalf ? 4 : 8, kSize = kHalf ? 2 : 4;
  uint32_t w[kWords];
  __device__ __forceinline__ uint32_t get(int j) const {
    return !kHalf ? w[j % kWords] : j % 2 ? w[(j / 2) % kWords] >> 16 : w[(j / 2) % kWords] & 0xFFFFu;
  }
  __device__ __forceinline__ void set(int j, uint32_t bits) {
    if (!kHalf) {
      w[j % kWords] = bits;
    } else {
      uint32_t& v = w[(j / 2) % kWords];
      v = j % 2 ? (v & 0xFFFFu) | (bits << 16) : (v & 0xFFFF0000u) | bits;
    }
  }
  // those of `which`, at logit `at` of the tensor (16-byte aligned)
  __device__ __forceinline__ void load(const void* p, long long at, uint32_t which) {
    if (which == 0xFFu) {
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * kSize);
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = from[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((which >> j) & 1u) set(j, kHalf ? static_cast<const uint16_t*>(p)[at + j] : static_cast<const uint32_t*>(p)[at + j]);
    }
  }
  __device__ __forceinline__ void store(void* p, long long at, uint32_t which) const {
    if (which == 0xFFu) {
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + at * kSize);
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (((which >> j) & 1u) == 0u) continue;
      if (kHalf) {
        static_cast<uint16_t*>(p)[at + j] = (uint16_t)get(j);
      } else {
        static_cast<uint32_t*>(p)[at + j] = get(j);
      }
    }
  }
};

// Rows of logits and out at the same place between 16-byte boundaries: kGroups
// groups of eight logits a thread, from the boundary before the row's start on.
template <int kType, int kThreads, int kGroups>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const AdjustParams p) {
  constexpr int kSpan = kThreads * 8 * kGroups;
  using G = Group<kType>;
  extern __shared__ uint4 s_words[];
  uint32_t* words = reinterpret_cast<uint32_t*>(s_words);
  __shared__ BiasList list;
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const splitk_adjust_t& h = p.how;
  const int row = (int)(blockIdx.x / (unsigned)p.spans), tid = (int)threadIdx.x;
  const long long in = (long long)row * p.stride, to = (long long)row * p.out_stride;
  const int past = (int)(((uintptr_t)p.logits + (uintptr_t)in * G::kSize) % 16) / G::kSize;   // the boundary
  const int lo = (int)(blockIdx.x % (unsigned)p.spans) * kSpan - past;
  const bool marked = h.history_length > 0 || h.bias_count > 0;
  const uint32_t* allowed =
      h.allowed ? reinterpret_cast<const uint32_t*>(h.allowed) + (long long)row * ((p.V + 31) / 32) : nullptr;

  uint32_t live[kGroups], keep[kGroups];                // within the row; allowed
  G x[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int e = lo + (g * kThreads + tid) * 8;
    live[g] = e >= p.V || e <= -8 ? 0u : (0xFFu << max(0, -e)) & (0xFFu >> max(0, e + 8 - p.V)) & 0xFFu;
    keep[g] = live[g] == 0u ? 0u : allowed ? live[g] & allowed_bits(allowed, e, p.V) : live[g];
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (keep[g] != 0u && !p.in_place) x[g].load(p.logits, in + lo + (g * kThreads + tid) * 8, live[g]);
  }
  const Changes changes(h, row);
  if (marked) mark<kThreads, kSpan>(h, row, lo, p.V, words, list);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int slot = (g * kThreads + tid) * 8;
    const long long e = (long long)lo + slot;
    uint32_t word[8] = {};
    if (marked && keep[g] != 0u) {
      const uint4 u = s_words[slot / 4], v = s_words[slot / 4 + 1];
      word[0] = u.x, word[1] = u.y, word[2] = u.z, word[3] = u.w, word[4] = v.x, word[5] = v.y, word[6] = v.z, word[7] = v.w;
    }
    const bool some = (word[0] | word[1] | word[2] | word[3] | word[4] | word[5] | word[6] | word[7]) != 0u;
    if (p.in_place) {
      if (!some && keep[g] == live[g]) continue;
      if (keep[g] != 0u) x[g].load(p.logits, in + e, live[g]);
    }
    if (some) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (word[j] != 0u) x[g].set(j, bits_of<kType>(changes.apply(value_of<kType>(x[g].get(j)), word[j], list, slot + j)));
      }
    }
    if (keep[g] != live[g]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (((keep[g] >> j) & 1u) == 0u) x[g].set(j, minus_infinity<kType>());
      }
    }
    if (live[g] != 0u) x[g].store(p.out, to + e, live[g]);
  }
}

// Rows at different places: a thread's logits are kThreads apart, so that a warp's
// accesses are consecutive.
template <int kType, int kThreads, int kEach>
__global__ void __launch_bounds__(kThreads) adjust_odd_kernel(const AdjustParams p) {
  constexpr int kSpan = kThreads * kEach;
  constexpr bool kHalf = kType != SPLITK_DTYPE_F32;
  extern __shared__ uint4 s_words[];
  uint32_t* words = reinterpret_cast<uint32_t*>(s_words);
  __shared__ BiasList list;
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const splitk_adjust_t& h = p.how;
  const int row = (int)(blockIdx.x / (unsigned)p.spans), tid = (int)threadIdx.x;
  const int lo = (int)(blockIdx.x % (unsigned)p.spans) * kSpan;
  const long long in = (long long)row * p.stride + lo, to = (long long)row * p.out_stride + lo;
  const bool marked = h.history_length > 0 || h.bias_count > 0;
  const uint32_t* allowed =
      h.allowed ? reinterpret_cast<const uint32_t*>(h.allowed) + (long long)row * ((p.V + 31) / 32) + lo / 32 : nullptr;
  uint32_t keep = 0u, x[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * kThreads + tid;
    const bool k = lo + e < p.V && (!allowed || ((allowed[e / 32] >> (e % 32)) & 1u) != 0u);
    keep |= (k ? 1u : 0u) << j;
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * kThreads + tid;
    x[j] = minus_infinity<kType>();
    if ((keep >> j) & 1u) x[j] = kHalf ? static_cast<const uint16_t*>(p.logits)[in + e] : static_cast<const uint32_t*>(p.logits)[in + e];
  }
  const Changes changes(h, row);
  if (marked) mark<kThreads, kSpan>(h, row, lo, p.V, words, list);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * kThreads + tid;
    if (lo + e >= p.V) continue;
    const uint32_t word = marked && ((keep >> j) & 1u) ? words[e] : 0u;
    if (word != 0u) x[j] = bits_of<kType>(changes.apply(value_of<kType>(x[j]), word, list, (uint32_t)e));
    if (kHalf) {
      static_cast<uint16_t*>(p.out)[to + e] = (uint16_t)x[j];
    } else {
      static_cast<uint32_t*>(p.out)[to + e] = x[j];
    }
  }
}

template <int kType, int kThreads, int kGroups>
cudaError_t launch_adjust(AdjustParams& p, int M, bool even, cudaStream_t stream) {
  constexpr int kSpan = kThreads * 8 * kGroups;
  const int past = even ? 16 / Group<kType>::kSize - 1 : 0;           // at most, before a row's start
  p.spans = (p.V + past + kSpan - 1) / kSpan;
  const bool marked = p.how.history_length > 0 || p.how.bias_count > 0;
  const size_t smem = marked ? (size_t)kSpan * 4 : 0;
  const dim3 grid((unsigned)((long long)M * p.spans));
  return even ? launch_chained(adjust_kernel<kType, kThreads, kGroups>, grid, dim3(kThreads), smem, 1, stream, p)
              : launch_chained(adjust_odd_kernel<kType, kThreads, 8 * kGroups>, grid, dim3(kThreads), smem, 1, stream, p);
}

template <int kType>
cudaError_t choose_adjust(AdjustParams& p, int M, bool even, int num_sms, cudaStream_t stream) {
  // long spans read the history fewer times; short ones fill the SMs
  const long long all = (long long)M * p.V;
  if (all <= (long long)num_sms * 4 * 2048) return launch_adjust<kType, 256, 1>(p, M, even, stream);
  return launch_adjust<kType, 256, 4>(p, M, even, stream);
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
  if (h.history_length < 0 || h.history_length > (1 << 29) || h.bias_count < 0 || h.bias_count > kMaxBias) {
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
  // a launch's CTAs, of at least 2048 logits
  if ((long long)M * (V / 2048 + 2) > 0x7FFFFFFFll) return SPLITK_ERR_INVALID_SHAPE;
  DeviceSize dev;
  const int rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  AdjustParams p{logits, stride, out_stride, out, h, V, 1, out == logits && stride == out_stride};
  // rows of both at the same place between 16-byte boundaries
  const bool even = ((uintptr_t)logits - (uintptr_t)out) % 16 == 0 && (stride - out_stride) * (long long)size % 16 == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = type == SPLITK_DTYPE_F32   ? choose_adjust<SPLITK_DTYPE_F32>(p, M, even, dev.num_sms, s)
                        : type == SPLITK_DTYPE_F16 ? choose_adjust<SPLITK_DTYPE_F16>(p, M, even, dev.num_sms, s)
                                                   : choose_adjust<SPLITK_DTYPE_BF16>(p, M, even, dev.num_sms, s);
  return launched(e);
}

}  // extern "C"
