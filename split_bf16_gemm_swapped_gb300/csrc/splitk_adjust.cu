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
// A CTA takes a span of one row's vocabulary: it counts those of the row's history
// that lie in the span in shared memory (whole numbers: any order gives the same)
// and applies them to the logits that its threads have loaded meanwhile.  Memory is
// the bound: each logit is read (but for eight banned ones in a row) and written
// once; the history is read once for each span, from L2.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "splitk.h"
#include "splitk_device.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

constexpr int kAdjustThreads = 256;
constexpr int kMaxBias = 1024;

struct AdjustParams {
  const void* logits;
  long long stride, out_stride;
  void* out;
  splitk_adjust_t how;
  int V, spans;
  bool vec;                 // 16-byte accesses to logits and out
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

// How a row's counted tokens change.
struct Penalties {
  float repetition, presence, frequency;
  bool any;
  __device__ __forceinline__ Penalties(const splitk_adjust_t& h, int row) {
    any = h.history != nullptr && (h.repetition != nullptr || h.presence != nullptr || h.frequency != nullptr);
    repetition = any && h.repetition ? h.repetition[row] : 1.0f;
    presence = any && h.presence ? h.presence[row] : 0.0f;
    frequency = any && h.frequency ? h.frequency[row] : 0.0f;
  }
  // word: 2 for each time behind the prompt, 1 more (once) for a token of the prompt
  __device__ __forceinline__ float apply(float x, uint32_t word) const {
    if (word == 0) return x;
    x = x > 0.0f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
    const uint32_t count = word >> 1;
    if (count != 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(frequency, (float)count)), presence);
    return x;
  }
};

// kGroups groups of eight logits a thread.  With `vec` a group is eight consecutive
// ones in 16-byte words; else a thread's logits are kAdjustThreads apart, so that a
// warp's accesses are consecutive whatever the alignment.
template <int kType, int kGroups, bool kVec>
__global__ void __launch_bounds__(kAdjustThreads) adjust_kernel(const AdjustParams p) {
  constexpr int kSpan = kAdjustThreads * 8 * kGroups;
  constexpr int kWords = kType == SPLITK_DTYPE_F32 ? 8 : 4;      // of a group
  extern __shared__ uint32_t s_count[];                 // [kSpan], then the biases [kSpan] where there are any
  float* s_bias = reinterpret_cast<float*>(s_count + kSpan);
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const splitk_adjust_t& h = p.how;
  const int tid = (int)threadIdx.x;
  const int row = (int)(blockIdx.x / (unsigned)p.spans), lo = (int)(blockIdx.x % (unsigned)p.spans) * kSpan;
  const int live = min(kSpan, p.V - lo);                // of the span
  const Penalties penalties(h, row);
  const bool biased = h.bias_count > 0;

  // which are banned, and the others' logits
  const uint32_t* allowed = h.allowed ? reinterpret_cast<const uint32_t*>(h.allowed) +
                                            (long long)row * ((p.V + 31) / 32) + lo / 32
                                      : nullptr;
  uint32_t keep[kGroups], w[kGroups][kVec ? kWords : 8];
  const long long in = (long long)row * p.stride + lo, to = (long long)row * p.out_stride + lo;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (kVec) {
      const int e = (g * kAdjustThreads + tid) * 8;
      keep[g] = e >= live ? 0u : allowed ? (allowed[e / 32] >> (e % 32)) & 0xFFu : 0xFFu;
    } else {
      keep[g] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = (g * 8 + j) * kAdjustThreads + tid;
        const bool k = e < live && (!allowed || ((allowed[e / 32] >> (e % 32)) & 1u) != 0u);
        keep[g] |= (k ? 1u : 0u) << j;
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (kVec) {
      // (V, or the vocabulary's end, need not be a multiple of eight: V of whole 16 bytes is)
      const int e = (g * kAdjustThreads + tid) * 8;
      if (keep[g] != 0u) {
        const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.logits) +
                                                           (in + e) * (kWords * 4 / 8));
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = from[i];
          w[g][4 * i] = v.x, w[g][4 * i + 1] = v.y, w[g][4 * i + 2] = v.z, w[g][4 * i + 3] = v.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = (g * 8 + j) * kAdjustThreads + tid;
        if ((keep[g] >> j) & 1u) {
          w[g][kVec ? 0 : j] = kType == SPLITK_DTYPE_F32 ? static_cast<const uint32_t*>(p.logits)[in + e]
                                                          : static_cast<const uint16_t*>(p.logits)[in + e];
        }
      }
    }
  }

  // the history's and the biases' tokens of the span
  if (penalties.any) {
    for (int i = tid; i < kSpan / 4; i += kAdjustThreads) reinterpret_cast<uint4*>(s_count)[i] = make_uint4(0, 0, 0, 0);
  }
  if (biased) {
    for (int i = tid; i < kSpan / 4; i += kAdjustThreads) reinterpret_cast<uint4*>(s_bias)[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  if (penalties.any) {
    const long long most = h.history_length;
    const long long n = h.lengths ? max(0ll, min(h.lengths[row], most)) : most;
    const long long prompt = h.prompt_lengths ? h.prompt_lengths[row] : 0;
    const long long* tokens = h.history + (long long)row * most;
    for (long long i = tid; i < n; i += kAdjustThreads) {
      const long long at = tokens[i] - lo;
      if (at < 0 || at >= live) continue;
      if (i >= prompt) {
        atomicAdd(&s_count[at], 2u);
      } else {
        atomicOr(&s_count[at], 1u);
      }
    }
  }
  if (biased) {
    // a token's biases are added in the list's order by the thread of the first
    const long long* ids = h.bias_ids + (long long)row * h.bias_count;
    const float* values = h.bias_values + (long long)row * h.bias_count;
    for (int b = tid; b < h.bias_count; b += kAdjustThreads) {
      const long long id = ids[b], at = id - lo;
      if (at < 0 || at >= live) continue;
      bool first = true;
      for (int c = 0; c < b; ++c) first = first && ids[c] != id;
      if (!first) continue;
      float sum = values[b];
      for (int c = b + 1; c < h.bias_count; ++c) {
        if (ids[c] == id) sum += values[c];
      }
      s_bias[at] = sum;
    }
  }
  __syncthreads();

#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = kVec ? (g * kAdjustThreads + tid) * 8 + j : (g * 8 + j) * kAdjustThreads + tid;
      const uint32_t bits = !kVec || kType == SPLITK_DTYPE_F32 ? w[g][j % (kVec ? kWords : 8)]
                            : j % 2                            ? w[g][(j / 2) % kWords] >> 16
                                                               : w[g][(j / 2) % kWords] & 0xFFFFu;
      o[j] = minus_infinity<kType>();
      if ((keep[g] >> j) & 1u) {
        float x = value_of<kType>(bits);
        if (penalties.any) x = penalties.apply(x, s_count[e]);
        if (biased) {
          const float b = s_bias[e];
          if (b != 0.0f) x = __fadd_rn(x, b);
        }
        o[j] = bits_of<kType>(x);
      }
    }
    if (kVec) {
      const int e = (g * kAdjustThreads + tid) * 8;
      if (e >= live) continue;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + (to + e) * (kWords * 4 / 8));
      if (kType == SPLITK_DTYPE_F32) {
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        dst[0] = make_uint4(o[0] | (o[1] << 16), o[2] | (o[3] << 16), o[4] | (o[5] << 16), o[6] | (o[7] << 16));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = (g * 8 + j) * kAdjustThreads + tid;
        if (e >= live) continue;
        if (kType == SPLITK_DTYPE_F32) {
          static_cast<uint32_t*>(p.out)[to + e] = o[j];
        } else {
          static_cast<uint16_t*>(p.out)[to + e] = (uint16_t)o[j];
        }
      }
    }
  }
}

template <int kType, int kGroups, bool kVec>
cudaError_t launch_adjust(AdjustParams& p, int M, cudaStream_t stream) {
  constexpr int kSpan = kAdjustThreads * 8 * kGroups;
  p.spans = (p.V + kSpan - 1) / kSpan;
  const size_t smem = (size_t)kSpan * 4 * (p.how.bias_count > 0 ? 2 : 1);
  return launch_chained(adjust_kernel<kType, kGroups, kVec>, dim3((unsigned)((long long)M * p.spans)), dim3(kAdjustThreads),
                        smem, 1, stream, p);
}

template <int kType, bool kVec>
cudaError_t choose_adjust(AdjustParams& p, int M, int num_sms, cudaStream_t stream) {
  // long spans read the history fewer times; short ones fill the SMs
  const long long all = (long long)M * p.V;
  if (all <= (long long)num_sms * 4 * 2048) return launch_adjust<kType, 1, kVec>(p, M, stream);
  return launch_adjust<kType, 2, kVec>(p, M, stream);
}

template <int kType>
cudaError_t choose_adjust(AdjustParams& p, int M, int num_sms, cudaStream_t stream) {
  return p.vec ? choose_adjust<kType, true>(p, M, num_sms, stream) : choose_adjust<kType, false>(p, M, num_sms, stream);
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
  if (h.history_length < 0 || h.history_length > (1 << 30) || h.bias_count < 0 || h.bias_count > kMaxBias) {
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
  if ((long long)M * ((V + 2047) / 2048) > 0x7FFFFFFFll) return SPLITK_ERR_INVALID_SHAPE;
  DeviceSize dev;
  const int rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  AdjustParams p{logits, stride, out_stride, out, h, V, 1, false};
  if (h.history_length == 0) p.how.history = nullptr;
  p.vec = V % 8 == 0 && aligned(logits, 16) && aligned(out, 16) && stride * (long long)size % 16 == 0 &&
          out_stride * (long long)size % 16 == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = type == SPLITK_DTYPE_F32   ? choose_adjust<SPLITK_DTYPE_F32>(p, M, dev.num_sms, s)
                        : type == SPLITK_DTYPE_F16 ? choose_adjust<SPLITK_DTYPE_F16>(p, M, dev.num_sms, s)
                                                   : choose_adjust<SPLITK_DTYPE_BF16>(p, M, dev.num_sms, s);
  return launched(e);
}

}  // extern "C"
