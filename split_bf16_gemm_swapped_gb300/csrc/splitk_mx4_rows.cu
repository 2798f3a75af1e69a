// Rows to microscaled 4-bit codes and back: splitk_quantize_mx4(),
// splitk_dequantize_mx4() and splitk_rmsnorm_mx4() (the format: splitk_mx4.cuh).
//
//   y = x + r                                   (f32; r' = y in r's type)
//   n = y w (1 / sqrt(mean(y^2) + eps))         (f32, in this order; quantise: n = x)
//   codes and scales of n
//
// A thread holds eight consecutive values (16 bytes of bf16) and four threads a
// block of 32, whose largest magnitude two exchanges of lanes give them all.
// Every byte is read and written once; memory is the bound: codes of 18432 x 7168 bf16
// 51.0 us and back 51.0 (6.6 TB/s, 98 % of a copy's rate), norm of 2048 x 7168 with an
// f32 residual 27.5 us (5.6 TB/s), of one row 2.3 us (launch and a chain of latencies).
// (Rows of 16416 to 32768 with an f32 residual spill some 550 bytes a thread: 512 x 32768 80.6 us.)
// Issue comes next: with 64-bit places and the largest magnitude in f32, codes took 93
// instructions a vector and 60 us.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"
#include "splitk_device.cuh"
#include "splitk_internal.h"
#include "splitk_mx4.cuh"

namespace splitk {

namespace {

constexpr int kVec = 8;

// Element types as the kernels' template arguments have them.
enum Kind : int { kNone = 0, kBf16 = 1, kF32 = 2, kF16 = 3 };

__host__ __device__ constexpr int size_of(int kind) { return kind == kF32 ? 4 : 2; }

__device__ __forceinline__ float f16_value(uint32_t bits) {
  float f;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(bits));
  return f;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int kKind>
__device__ __forceinline__ float half_value(uint32_t bits) {
  return kKind == kF16 ? f16_value(bits) : __uint_as_float(bits << 16);
}
template <int kKind>
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  return kKind == kF16 ? pack_f16x2(lo, hi) : dev::pack_bf16x2(lo, hi);
}

// Both halves' larger ones.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight consecutive elements, in 16-byte words or (`vec` false) one by one.
template <int kKind>
struct Eight {
  static constexpr int kWords = kKind == kF32 ? 8 : 4;
  uint32_t w[kWords];
  template <class Place>
  __device__ __forceinline__ void load(const void* p, Place at, bool vec) {
    if (vec) {
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * size_of(kKind));
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = from[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if (kKind == kF32) {
      const uint32_t* from = static_cast<const uint32_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = from[i];
    } else {
      const uint16_t* from = static_cast<const uint16_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = (uint32_t)from[2 * i] | ((uint32_t)from[2 * i + 1] << 16);
    }
  }
  __device__ __forceinline__ void values(float (&v)[kVec]) const {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      v[j] = kKind == kF32 ? __uint_as_float(w[j % kWords]) : half_value<kKind>(j % 2 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu);
    }
  }
  // The largest magnitude of a block (four lanes' vectors), from the bits: without
  // their signs the values are ordered as whole numbers, NaN above infinity.
  __device__ __forceinline__ float block_top() const {
    constexpr uint32_t kMagnitude = kKind == kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    const auto larger = [](uint32_t a, uint32_t b) { return kKind == kF32 ? max(a, b) : max_u16x2(a, b); };
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) top = larger(top, w[i] & kMagnitude);
    top = larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    return kKind == kF32 ? __uint_as_float(top) : half_value<kKind>(max(top & 0xFFFFu, top >> 16));
  }
  __device__ __forceinline__ void set(const float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      w[i] = kKind == kF32 ? __float_as_uint(v[i]) : pack_half2<kKind>(v[(2 * i) % kVec], v[(2 * i + 1) % kVec]);
    }
  }
  __device__ __forceinline__ void store(void* p, long long at, bool vec) const {
    if (vec) {
      uint4* to = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p) + at * size_of(kKind));
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if (kKind == kF32) {
      uint32_t* to = static_cast<uint32_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < kWords; ++i) to[i] = w[i];
    } else {
      uint16_t* to = static_cast<uint16_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < kWords; ++i) to[2 * i] = (uint16_t)(w[i] & 0xFFFFu), to[2 * i + 1] = (uint16_t)(w[i] >> 16);
    }
  }
};

// max that keeps a NaN of either operand.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The codes of eight values of a block whose largest magnitude is `top`, and its
// scale code.
__device__ __forceinline__ uint32_t codes_of(const float (&n)[kVec], float top, uint32_t& code) {
  code = mx_scale_code(top);
  const float inverse = mx_inverse_scale(code);
  float q[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) q[j] = n[j] * inverse;
  return code == kMxNaN ? 0u : dev::e2m1x8(q);
}

// The same for four lanes to a block: all lanes of the warp call it.
__device__ __forceinline__ uint32_t block_codes(const float (&n)[kVec], uint32_t& code) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < kVec; ++j) top = max_nan(top, fabsf(n[j]));
  top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  return codes_of(n, top, code);
}

// ---------------------------------------------------------------- quantise
struct QuantizeParams {
  const void* x;
  long long x_stride;       // elements between rows
  uint8_t* codes;           // [rows][width / 2]
  uint8_t* scale;           // [rows][width / 32]
  long long rows, width;
  uint32_t chunks;          // of a row, `step` vectors of kEach threads
  bool vec;
};

constexpr int kRowThreads = 256;
constexpr int kEach = 4;                       // vectors a thread holds

// A CTA takes blockDim.y rows, kEach * blockDim.x vectors of each.
template <int kKind>
__global__ void __launch_bounds__(kRowThreads) quantize_kernel(const QuantizeParams p) {
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const uint32_t group = p.chunks == gridDim.x ? 0u : blockIdx.x / p.chunks, chunk = blockIdx.x - group * p.chunks;
  const long long row = (long long)group * blockDim.y + threadIdx.y;
  const long long first = (long long)chunk * (kEach * blockDim.x * kVec);
  // from the CTA's part of the row on, 32 bits hold a place
  const int left = row < p.rows ? (int)min(p.width - first, (long long)(kEach * kRowThreads * kVec)) : 0;
  const int step = (int)blockDim.x * kVec, at = (int)threadIdx.x * kVec;
  const uint8_t* from = static_cast<const uint8_t*>(p.x) + (row * p.x_stride + first) * size_of(kKind);
  uint8_t* codes = p.codes + (row * p.width + first) / 2;
  uint8_t* scale = p.scale + (row * p.width + first) / kMxBlock;
  Eight<kKind> e[kEach] = {};
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (at + i * step < left) e[i].load(from, at + i * step, p.vec);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int place = at + i * step;
    const float top = e[i].block_top();
    if (place >= left) continue;                       // (the same in a block's four lanes)
    float v[kVec];
    e[i].values(v);
    uint32_t code;
    const uint32_t q = codes_of(v, top, code);
    *reinterpret_cast<uint32_t*>(codes + (uint32_t)place / 2u) = q;
    if (threadIdx.x % 4 == 0) scale[(uint32_t)place / (uint32_t)kMxBlock] = (uint8_t)code;
  }
}

// ---------------------------------------------------------------- dequantise
// Eight codes of a thread at a time, whole blocks of a thread group as above.
template <int kKind>
__global__ void __launch_bounds__(kRowThreads) dequantize_kernel(const uint8_t* codes, const uint8_t* scale, void* out,
                                                                 long long vectors) {
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const long long first = (long long)blockIdx.x * (kEach * kRowThreads) + threadIdx.x;
  uint32_t w[kEach], s[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const long long at = first + i * kRowThreads;
    w[i] = at < vectors ? reinterpret_cast<const uint32_t*>(codes)[at] : 0u;
    s[i] = at < vectors ? scale[at / 4] : 0u;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const long long at = first + i * kRowThreads;
    if (at >= vectors) continue;
    const float by = mx_scale(s[i]);
    float v[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      // sign, and the magnitude's two exponent bits and one fraction bit over
      // f32's: worth x 2^-126 (a zero exponent field is f32's subnormal), times 2^126
      const uint32_t c = w[i] >> (4 * j);
      v[j] = __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * 0x1p126f * by;
    }
    Eight<kKind> o;
    o.set(v);
    o.store(out, at * kVec, true);
  }
}

// ---------------------------------------------------------------- norm
constexpr int kMaxRowThreads = 1024;

struct NormParams {
  const void* x;            // bf16 [rows][x_stride]
  long long x_stride;
  const void* residual;     // bf16 or f32 [rows][width], or null
  void* residual_out;
  const void* weight;       // bf16 or f32 [width]
  float mean_of;            // 1 / width
  float eps;
  uint8_t* codes;
  uint8_t* scale;
  int rows, width;
  bool x_vec, vec;          // 16-byte accesses to x; to the others
};

// A sum of squares as a whole number of 2^-shift.
struct FixedSum {
  uint32_t units;           // at most 2^31
  float rest;               // of a unit: what a join of sums cut off below one
  int shift;                // kBadShift: an addend was NaN or infinite
};
constexpr int kBadShift = -1024, kNoShift = 1024;       // (finite sums: -102 .. 151)

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// v 2^e for |e| up to 252, in two factors that are normal numbers.
__device__ __forceinline__ float scaled(float v, int e) { return v * power_of_two(e >> 1) * power_of_two(e - (e >> 1)); }

// The sum over a warp of values >= 0, each rounded to the unit that lets the largest
// have 26 bits: exact but for those roundings, whatever the order, in two
// reductions of whole numbers (in f64, which has two lanes an SM, a row of 7168
// took twice as long as its memory).
__device__ __forceinline__ FixedSum warp_sum(float v) {
  const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));        // (NaN of either sign is above all)
  const bool bad = top >= 0x7F800000u;
  const int shift = 25 - ((int)max(top >> 23, 1u) - 127);
  const int units = __reduce_add_sync(0xFFFFFFFFu, bad ? 0 : __float2int_rn(scaled(v, shift)));
  return {(uint32_t)units, 0.0f, bad ? kBadShift : shift};
}

// The sum of up to 32 warps' sums, one a lane (kNoShift in the others): in units of 32
// of the coarsest, and 27 bits below them, so nothing is cut off of a sum whose own unit
// is 2^-22 of the coarsest or more.  (With each warp's 31 bits passed on as an f32 value, 24
// rows in a hundred of 1024 f32 values had another mean, now 6.)
__device__ __forceinline__ FixedSum join_sums(uint32_t units, int shift) {
  const int coarsest = __reduce_min_sync(0xFFFFFFFFu, shift);
  const unsigned long long w = ((unsigned long long)units << 32) >> min(shift - coarsest + 5, 63);
  const uint32_t whole = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)(w >> 32));
  const uint32_t rest = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)w >> 5);
  return {whole, (float)rest * 0x1p-27f, coarsest == kBadShift ? kBadShift : coarsest - 5};
}

// 1 / sqrt(mean + eps) of the row, in every thread of it, from the threads' own sums
// of 8 to 32 squares, which are f32 and the one thing that rounds on the way: the mean
// does not depend on the order of additions.  By a model of this arithmetic, rows of
// normal values whose mean is not the exact one rounded to f32, but its neighbour, are 2 in
// a hundred at 7168 with an f32 residual, 4 to 6 at 1024 and 2048, 8 to 25 up to 512, and 9
// to 22 with values of bf16 (28 to 43 above 16384, a thread's 32 squares).  A row is one warp
// (blockDim.x = 32) or the whole CTA, which takes turns between two buffers.  NaN for a row
// whose sum passes f32.
__device__ __forceinline__ float row_factor(const NormParams& p, float own, int turn) {
  FixedSum s = warp_sum(own);
  if (blockDim.x != 32) {
    __shared__ int2 s_sum[2][32];
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, warps = (int)blockDim.x >> 5;
    if (lane == 0) s_sum[turn][warp] = make_int2((int)s.units, s.shift);
    __syncthreads();
    const int2 one = lane < warps ? s_sum[turn][lane] : make_int2(0, kNoShift);
    s = join_sums((uint32_t)one.x, one.y);
  }
  const bool bad = s.shift == kBadShift;
  const int shift = bad ? 0 : s.shift;
  // units 2^-shift / width, as the f32 quotient and what it leaves
  const float hi = __uint2float_rz(s.units), lo = (float)(s.units - (uint32_t)hi) + s.rest;
  const float inverse = p.mean_of, width = (float)p.width;
  const float q = hi * inverse, mean = q + (fmaf(-q, width, hi) + lo) * inverse;
  const float factor = 1.0f / sqrtf(scaled(mean, -shift) + p.eps);
  const bool past = bad || !(scaled(hi, -shift) <= 3.4028234e38f);
  return past ? __uint_as_float(0x7FC00000u) : factor;
}

// Values n of a thread's vector from y w: codes and scale stored.
__device__ __forceinline__ void store_codes(const NormParams& p, long long at, bool in, float (&z)[kVec], float factor) {
#pragma unroll
  for (int j = 0; j < kVec; ++j) z[j] *= factor;
  uint32_t code;
  const uint32_t q = block_codes(z, code);
  if (!in) return;
  *reinterpret_cast<uint32_t*>(p.codes + at / 2) = q;
  if (threadIdx.x % 4 == 0) p.scale[at / kMxBlock] = (uint8_t)code;
}

// y of a vector (and its sum with the residual written), the squares' sum, y w.
template <int kRes, int kW>
__device__ __forceinline__ void norm_vector(const NormParams& p, const Eight<kBf16>& x, const Eight<kRes ? kRes : 1>& r,
                                            long long base, int e, bool write, float (&z)[kVec], float& sum) {
  x.values(z);
  if (kRes != kNone) {
    float rv[kVec];
    r.values(rv);
#pragma unroll
    for (int j = 0; j < kVec; ++j) z[j] += rv[j];
    if (write) {
      Eight<kRes ? kRes : 1> o;
      o.set(z);
      o.store(p.residual_out, base + e, p.vec);
    }
  }
  Eight<kW> ww;
  float w[kVec];
  ww.load(p.weight, e, p.vec);
  ww.values(w);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    sum = fmaf(z[j], z[j], sum);
    z[j] *= w[j];
  }
}

// kVecs vectors a thread, rows of up to 8 * kVecs * 1024.  A CTA takes row after
// row; the next row's words are on their way while this one is reduced and coded.
template <int kRes, int kW, int kVecs>
__global__ void __launch_bounds__(kMaxRowThreads) norm_kernel(const NormParams p) {
  constexpr bool kNext = kVecs <= 2;     // registers for the next row's words
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const int tid = (int)threadIdx.x, step = (int)blockDim.x, stride = (int)(gridDim.x * blockDim.y);
  Eight<kBf16> xw[kVecs];
  Eight<kRes ? kRes : 1> rw[kVecs];
  const auto load = [&](int row) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = (v * step + tid) * kVec;
      if (e >= p.width) continue;
      xw[v].load(p.x, (long long)row * p.x_stride + e, p.x_vec);
      if (kRes != kNone) rw[v].load(p.residual, (long long)row * p.width + e, p.vec);
    }
  };
  int row = (int)(blockIdx.x * blockDim.y + threadIdx.y);
  if (row < p.rows) load(row);
  for (int turn = 0; row < p.rows; row += stride, turn ^= 1) {     // uniform in a row's threads
    const long long base = (long long)row * p.width;
    float z[kVecs][kVec] = {};
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = (v * step + tid) * kVec;
      if (e < p.width) norm_vector<kRes, kW>(p, xw[v], rw[v], base, e, true, z[v], sum);
    }
    if (kNext && row + stride < p.rows) load(row + stride);
    const float factor = row_factor(p, sum, turn);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = (v * step + tid) * kVec;
      store_codes(p, base + e, e < p.width, z[v], factor);
    }
    if (!kNext && row + stride < p.rows) load(row + stride);
  }
}

// Rows wider than a CTA's registers hold are read twice.  The first pass writes
// nothing, so the residual may be updated in place: each thread's second pass
// reads an element before it writes it.
template <int kRes, int kW>
__global__ void __launch_bounds__(kMaxRowThreads) long_norm_kernel(const NormParams p) {
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const int row = (int)blockIdx.x, step = (int)blockDim.x * kVec;
  const long long base = (long long)row * p.width;
  float z[kVec], sum = 0.0f, factor = 0.0f;
  Eight<kBf16> x;
  Eight<kRes ? kRes : 1> r;
  for (int pass = 0; pass < 2; ++pass) {
    float low = 0.0f;                                   // what the thread's sum has lost (Kahan 1965)
    for (long long first = 0; first < p.width; first += step) {    // uniform: the blocks' lanes stay together
      const long long e = first + threadIdx.x * kVec;
      const bool in = e < p.width;
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) z[j] = 0.0f;
      if (in) {
        x.load(p.x, (long long)row * p.x_stride + e, p.x_vec);
        if (kRes != kNone) r.load(p.residual, base + e, p.vec);
        norm_vector<kRes, kW>(p, x, r, base, (int)e, pass == 1, z, part);
      }
      if (pass == 0) {
        const float add = __fsub_rn(part, low), next = __fadd_rn(sum, add);
        low = __fsub_rn(__fsub_rn(next, sum), add);
        sum = next;
      } else {
        store_codes(p, base + e, in, z, factor);
      }
    }
    if (pass == 0) factor = row_factor(p, sum, 0);
  }
}

template <int kRes, int kW>
cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int vecs = p.width / kVec;
  if (vecs > 4 * kMaxRowThreads) {
    return launch_chained(long_norm_kernel<kRes, kW>, dim3((unsigned)p.rows), dim3(kMaxRowThreads), 0, 1, stream, p);
  }
  const auto threads = [&](int per) { return (unsigned)(((vecs + per - 1) / per + 31) & ~31); };
  // A warp a row of up to 512 features, four rows a CTA; else a CTA a row.  Few
  // rows get one vector a thread, for the shortest chain of latencies; many get
  // two and a CTA takes several.
  const bool warp_rows = vecs <= 64;
  const bool few = p.rows <= 2 * num_sms;
  const int per = warp_rows ? (vecs <= 32 ? 1 : 2) : vecs > 2 * kMaxRowThreads ? 4 : few && vecs <= kMaxRowThreads ? 1 : 2;
  const dim3 block = warp_rows ? dim3(32, 4) : dim3(threads(per));
  // as many CTAs as are resident at once (64 registers a thread: 1024 threads an SM)
  const int resident = num_sms * (kMaxRowThreads / (int)(block.x * block.y));
  const int ctas = (p.rows + (int)block.y - 1) / (int)block.y;
  const dim3 grid((unsigned)(ctas < resident ? ctas : resident));
  if (per == 1) return launch_chained(norm_kernel<kRes, kW, 1>, grid, block, 0, 1, stream, p);
  if (per == 2) return launch_chained(norm_kernel<kRes, kW, 2>, grid, block, 0, 1, stream, p);
  return launch_chained(norm_kernel<kRes, kW, 4>, grid, block, 0, 1, stream, p);
}

template <int kRes>
cudaError_t launch_weight(const NormParams& p, int weight_type, int num_sms, cudaStream_t stream) {
  return weight_type == SPLITK_DTYPE_F32 ? launch_norm<kRes, kF32>(p, num_sms, stream)
                                         : launch_norm<kRes, kBf16>(p, num_sms, stream);
}

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }
inline bool known_type(int t) { return t == SPLITK_DTYPE_BF16 || t == SPLITK_DTYPE_F32 || t == SPLITK_DTYPE_F16; }
inline uintptr_t type_size(int t) { return t == SPLITK_DTYPE_F32 ? 4u : 2u; }

constexpr long long kMost = 1ll << 30;         // rows, and their width

int check_shape(long long M, long long K) {
  return M < 1 || K < 1 || K % kMxBlock != 0 || M > kMost || K > kMost ? SPLITK_ERR_INVALID_SHAPE : SPLITK_OK;
}

}  // namespace

}  // namespace splitk

using namespace splitk;

extern "C" {

SPLITK_API int splitk_quantize_mx4(const void* x, int x_type, long long x_stride, void* codes, void* scale, int M, int K,
                                   splitk_stream_t stream) {
  if (!x || !codes || !scale) return SPLITK_ERR_NULL;
  if (!known_type(x_type)) return SPLITK_ERR_INVALID_ARGUMENT;
  int rc = check_shape(M, K);
  if (rc != SPLITK_OK || x_stride < K) return SPLITK_ERR_INVALID_SHAPE;
  if (!aligned(x, type_size(x_type)) || !aligned(codes, 16)) return SPLITK_ERR_MISALIGNED;
  QuantizeParams p{x, x_stride, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scale), M, K, 1u, false};
  p.vec = aligned(x, 16) && x_stride * (long long)type_size(x_type) % 16 == 0;
  if (x_stride == K) p.rows = 1, p.width = (long long)M * K, p.x_stride = p.width;     // one row of all
  // rows of fewer vectors than a CTA's threads share it
  const long long vecs = p.width / kVec;
  unsigned wide = 32;
  while (wide < kRowThreads && (long long)wide * kEach < vecs) wide *= 2;
  const dim3 block(wide, kRowThreads / wide);
  const long long chunks = (vecs + (long long)kEach * wide - 1) / ((long long)kEach * wide);
  const long long ctas = (p.rows + block.y - 1) / block.y * chunks;
  if (ctas > 0x7FFFFFFFll) return SPLITK_ERR_INVALID_SHAPE;
  p.chunks = (uint32_t)chunks;
  DeviceSize dev;
  rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  const dim3 grid((unsigned)ctas);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (x_type) {
    case SPLITK_DTYPE_F32: return launched(launch_chained(quantize_kernel<kF32>, grid, block, 0, 1, s, p));
    case SPLITK_DTYPE_F16: return launched(launch_chained(quantize_kernel<kF16>, grid, block, 0, 1, s, p));
    default: return launched(launch_chained(quantize_kernel<kBf16>, grid, block, 0, 1, s, p));
  }
}

SPLITK_API int splitk_dequantize_mx4(const void* codes, const void* scale, void* out, int out_type, int M, int K,
                                     splitk_stream_t stream) {
  if (!codes || !scale || !out) return SPLITK_ERR_NULL;
  if (!known_type(out_type)) return SPLITK_ERR_INVALID_ARGUMENT;
  int rc = check_shape(M, K);
  if (rc != SPLITK_OK) return rc;
  if (!aligned(codes, 16) || !aligned(out, 16)) return SPLITK_ERR_MISALIGNED;
  const long long vectors = (long long)M * K / kVec;
  const long long ctas = (vectors + kEach * kRowThreads - 1) / (kEach * kRowThreads);
  if (ctas > 0x7FFFFFFFll) return SPLITK_ERR_INVALID_SHAPE;
  DeviceSize dev;
  rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  const dim3 grid((unsigned)ctas), block(kRowThreads);
  const uint8_t *c = static_cast<const uint8_t*>(codes), *sc = static_cast<const uint8_t*>(scale);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (out_type) {
    case SPLITK_DTYPE_F32: return launched(launch_chained(dequantize_kernel<kF32>, grid, block, 0, 1, s, c, sc, out, vectors));
    case SPLITK_DTYPE_F16: return launched(launch_chained(dequantize_kernel<kF16>, grid, block, 0, 1, s, c, sc, out, vectors));
    default: return launched(launch_chained(dequantize_kernel<kBf16>, grid, block, 0, 1, s, c, sc, out, vectors));
  }
}

SPLITK_API int splitk_rmsnorm_mx4(const void* x, long long x_stride, const void* residual, void* residual_out,
                                  int residual_type, const void* weight, int weight_type, float eps, void* codes,
                                  void* scale, int M, int D, splitk_stream_t stream) {
  if (!x || !codes || !scale || !weight || (residual != nullptr) != (residual_out != nullptr)) return SPLITK_ERR_NULL;
  int rc = check_shape(M, D);
  if (rc != SPLITK_OK || x_stride < D) return SPLITK_ERR_INVALID_SHAPE;
  if (!(eps > 0.0f) || !(eps <= 3.4e38f)) return SPLITK_ERR_INVALID_ARGUMENT;
  if (weight_type != SPLITK_DTYPE_BF16 && weight_type != SPLITK_DTYPE_F32) return SPLITK_ERR_INVALID_ARGUMENT;
  if (residual && residual_type != SPLITK_DTYPE_BF16 && residual_type != SPLITK_DTYPE_F32) {
    return SPLITK_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(x, 2) || !aligned(codes, 16) || !aligned(weight, type_size(weight_type))) return SPLITK_ERR_MISALIGNED;
  if (residual && (!aligned(residual, type_size(residual_type)) || !aligned(residual_out, type_size(residual_type)))) {
    return SPLITK_ERR_MISALIGNED;
  }
  DeviceSize dev;
  rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  const NormParams p{x, x_stride, residual, residual_out, weight, 1.0f / (float)D, eps, static_cast<uint8_t*>(codes),
                     static_cast<uint8_t*>(scale), M, D, aligned(x, 16) && x_stride % kVec == 0,
                     aligned(weight, 16) && aligned(residual, 16) && aligned(residual_out, 16)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = !residual                               ? launch_weight<kNone>(p, weight_type, dev.num_sms, s)
                        : residual_type == SPLITK_DTYPE_F32 ? launch_weight<kF32>(p, weight_type, dev.num_sms, s)
                                                                : launch_weight<kBf16>(p, weight_type, dev.num_sms, s);
  return launched(e);
}

}  // extern "C"
