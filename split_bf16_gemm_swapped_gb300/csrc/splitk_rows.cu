// Activations to 8-bit codes, a row (token) at a time: splitk_rmsnorm_i8()
// and splitk_quantize_i8().
//
//   y = x + r                                   (f32; r' = y in r's type)
//   n = y * w / sqrt(mean(y^2) + eps)           (quantise alone: n = x)
//   s = max(max|n| (1/127), 2^-126);  q = rne(n / s), the f32 quotient
//
// max|n| = max|y w| / rms, so one joint reduction of (sum y^2, max|y w|) over
// the row gives both statistics, and the row's values z = y w stay on
// chip between reading and coding: every byte is read and written once (up to
// 32768 features; longer rows are read twice, long_rows_kernel), and memory is
// the bound (2048 x 7168 with a bf16 residual 16.8 us, 92 % of the copy
// rate; 18432 x 7168 codes 74 us, 80 %).  Up to 16384 features in vectors they stay in
// registers; with four vectors a thread some spill (a thread's bytes: 30 at most
// without a residual, 260-310 with one: 64 x 20000 6.4 us, 1.3 the copy's), and so they
// do in odd_rows_kernel (50-90).  Sums and statistics are f32; a code is
// rounded by adding 1.5 * 2^23 (the sum's low byte is then the two's complement
// code, rounded to nearest even).

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"
#include "splitk_device.cuh"
#include "splitk_internal.h"

namespace splitk {

namespace {

constexpr float kMinScale = 1.17549435e-38f;   // 2^-126, the smallest normal f32
constexpr float kMaxF32 = 3.40282347e38f;
constexpr int kMaxRowThreads = 1024;
constexpr int kVec = 8;                        // elements of one 16-byte load of bf16

struct RowParams {
  const uint16_t* x;        // bf16 [rows][x_stride]
  long long x_stride;
  const void* residual;     // bf16 or f32 [rows][width], or null
  void* residual_out;
  const void* weight;       // bf16 or f32 [width]
  float eps;
  int8_t* q;                // [rows][width]
  float* scale;             // [rows]
  int rows, width;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_one(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// max that keeps a NaN of either operand (a row holding one must not come
// out as finite codes).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The code of n, rne(n / s) with the f32 quotient (|n / s| <= 127), in the low
// byte.  Values at and beside halves between two codes are common in bf16 rows (half
// the largest is one), and the product with r = 1 / s alone sends them either way.
// The product's remainder n - q s (exact in one fused operation) times r
// corrects it to the quotient (Markstein 1990, "Computation of elementary functions
// on the IBM RISC System/6000 processor"), for two more instructions on a pair.
constexpr float kRound = 12582912.0f;          // 1.5 * 2^23
__device__ __forceinline__ uint32_t code_of(float n, float s, float r) {
  const float q = __fmul_rn(n, r);
  return __float_as_uint(__fadd_rn(fmaf(fmaf(-q, s, n), r, q), kRound));
}

__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return dev::prmt(dev::prmt(a, b, 0x0040u), dev::prmt(c, d, 0x0040u), 0x5410u);
}

// Eight of them, two in an instruction.
__device__ __forceinline__ uint2 codes_of(const float (&n)[kVec], float s, float r) {
  const uint64_t minus_s = dev::f32x2(-s, -s), rr = dev::f32x2(r, r), round = dev::f32x2(kRound, kRound);
  uint32_t c[kVec];
#pragma unroll
  for (int j = 0; j < kVec; j += 2) {
    const uint64_t v = dev::f32x2(n[j], n[j + 1]), q = dev::f32x2_mul(v, rr);
    float lo, hi;
    dev::f32x2_split(dev::f32x2_add(dev::f32x2_fma(dev::f32x2_fma(q, minus_s, v), rr, q), round), lo, hi);
    c[j] = __float_as_uint(lo), c[j + 1] = __float_as_uint(hi);
  }
  return make_uint2(pack_codes(c[0], c[1], c[2], c[3]), pack_codes(c[4], c[5], c[6], c[7]));
}

// Eight consecutive elements in 16-byte words of type kType (1 bf16, 2 f32).
template <int kType>
struct Words {
  uint4 w[kType];
  __device__ __forceinline__ void load(const void* p, long long at) {
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (2 * kType));
#pragma unroll
    for (int i = 0; i < kType; ++i) w[i] = from[i];
  }
  __device__ __forceinline__ void unpack(float (&v)[kVec]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      v[j] = kType == 2 ? __uint_as_float(u[j]) : j % 2 == 0 ? bf16_lo(u[j / 2]) : bf16_hi(u[j / 2]);
    }
  }
};

template <int kType>
__device__ __forceinline__ float load1(const void* p, long long at) {
  return kType == 1 ? bf16_one(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

template <int kType>
__device__ __forceinline__ void store1(void* p, long long at, float v) {
  if (kType == 1) {
    static_cast<uint16_t*>(p)[at] = (uint16_t)(dev::pack_bf16x2(v, 0.0f) & 0xFFFFu);
  } else {
    static_cast<float*>(p)[at] = v;
  }
}

// The row's sum and maximum, in every thread of the row.  A row is one warp
// (blockDim.x = 32, blockDim.y rows a CTA) or the whole CTA, which takes turns
// between two buffers so that one barrier a row is enough.
__device__ __forceinline__ void reduce_row(float& sum, float& amax, int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  }
  if (blockDim.x == 32) return;
  __shared__ float s_sum[2][32], s_max[2][32];
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, warps = (int)blockDim.x >> 5;
  if (lane == 0) s_sum[turn][warp] = sum, s_max[turn][warp] = amax;
  __syncthreads();
  sum = lane < warps ? s_sum[turn][lane] : 0.0f;
  amax = lane < warps ? s_max[turn][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  }
}

// The row's scale, and what its codes are made of: values z = y w become
// n = z * factor (factor 1 where there is no norm), and n's code is that of n / s,
// r = 1 / s.  (n and s are both 2^64 times themselves where s is so small that a
// remainder would pass f32's smallest numbers; a quotient's the same.)
//
// 1 / 127 is a factor, as PyTorch's division of a GPU tensor by 127 has it: codes
// and scales are to the bit what the elementary operations give for a row.  A row
// that holds a NaN or an infinity (or whose sum of squares or largest n passes
// f32) has no codes: its scale is NaN, and so is every product that uses it.
struct RowCodes {
  float scale, factor, lift, s, r;
  __device__ __forceinline__ RowCodes(bool norm, float sum, float amax, int width, float eps) {
    factor = norm ? 1.0f / sqrtf(sum / (float)width + eps) : 1.0f;
    const float top = amax * factor;               // max|n|: rounding keeps the order
    scale = fmaxf(top * (1.0f / 127.0f), kMinScale);
    lift = scale < 0x1p-60f ? 0x1p64f : 1.0f;
    s = scale * lift;
    r = 1.0f / s;
    if (!(sum <= kMaxF32) || !(top <= kMaxF32)) scale = __uint_as_float(0x7FC00000u);
  }
};

// kRes: 0 no residual, 1 bf16, 2 f32.  kW: 0 no norm (quantise alone), 1 bf16
// weight, 2 f32 weight.  kVecs: 8-element vectors a thread holds.
//
// Rows and weight in 16-byte vectors.  A CTA takes row after row; the next row's
// words are on their way while this one is reduced and coded, so that loads are
// in flight all the time (18432 x 7168 codes, a CTA a row: 103 us, so 74).
template <int kRes, int kW, int kVecs>
__global__ void __launch_bounds__(kMaxRowThreads) rows_kernel(const RowParams p) {
  constexpr bool kNext = kVecs <= 2;     // registers for the next row's words
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const int tid = (int)threadIdx.x, step = (int)blockDim.x, stride = (int)(gridDim.x * blockDim.y);
  Words<1> xw[kVecs];
  Words<kRes == 0 ? 1 : kRes> rw[kVecs];
  const auto load = [&](int row) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = (v * step + tid) * kVec;
      if (e >= p.width) continue;
      xw[v].load(p.x, (long long)row * p.x_stride + e);
      if (kRes != 0) rw[v].load(p.residual, (long long)row * p.width + e);
    }
  };
  int row = (int)(blockIdx.x * blockDim.y + threadIdx.y);
  if (row < p.rows) load(row);
  for (int turn = 0; row < p.rows; row += stride, turn ^= 1) {     // uniform in a row's threads
    const long long base = (long long)row * p.width;
    float z[kVecs][kVec];
    float sum = 0.0f, amax = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = (v * step + tid) * kVec;
#pragma unroll
      for (int j = 0; j < kVec; ++j) z[v][j] = 0.0f;
      if (e >= p.width) continue;
      xw[v].unpack(z[v]);
      if (kRes != 0) {
        float r[kVec];
        rw[v].unpack(r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) z[v][j] += r[j];
        if (kRes == 1) {
          uint4 o;
          o.x = dev::pack_bf16x2(z[v][0], z[v][1]), o.y = dev::pack_bf16x2(z[v][2], z[v][3]);
          o.z = dev::pack_bf16x2(z[v][4], z[v][5]), o.w = dev::pack_bf16x2(z[v][6], z[v][7]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + base + e) = o;
        } else {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + base + e);
          o[0] = make_float4(z[v][0], z[v][1], z[v][2], z[v][3]);
          o[1] = make_float4(z[v][4], z[v][5], z[v][6], z[v][7]);
        }
      }
      if (kW != 0) {
        Words<kW == 0 ? 1 : kW> ww;
        float w[kVec];
        ww.load(p.weight, e);
        ww.unpack(w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          sum = fmaf(z[v][j], z[v][j], sum);
          z[v][j] *= w[j];
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) amax = max_nan(amax, fabsf(z[v][j]));
    }
    if (kNext && row + stride < p.rows) load(row + stride);
    reduce_row(sum, amax, turn);
    const RowCodes codes(kW != 0, sum, amax, p.width, p.eps);
    if (tid == 0) p.scale[row] = codes.scale;
    if (kW != 0) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) z[v][j] *= codes.factor;
      }
    }
    if (codes.lift != 1.0f) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) z[v][j] *= codes.lift;
      }
    }
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = (v * step + tid) * kVec;
      if (e >= p.width) continue;
      *reinterpret_cast<uint2*>(p.q + base + e) = codes_of(z[v], codes.s, codes.r);
    }
    if (!kNext && row + stride < p.rows) load(row + stride);
  }
}

// Rows of any width and alignment, an element at a time (lane by lane, so that
// a warp's loads are consecutive), kEach of them a thread.  With a residual two
// thousand threads an SM (32 registers) serve better than half as many: 333 x 4999,
// f32, 8.9 us and 11.6, spills of 52 bytes included; without one the loads want the registers: 2000 x 5001 codes
// 20 us and 17.
template <int kRes, int kW, int kEach>
__global__ void __launch_bounds__(kMaxRowThreads, kRes != 0 && kEach == 8 ? 2 : 1) odd_rows_kernel(const RowParams p) {
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const int row = (int)blockIdx.x, tid = (int)threadIdx.x, step = (int)blockDim.x;
  const uint16_t* x = p.x + (long long)row * p.x_stride;
  const long long base = (long long)row * p.width;
  float z[kEach];
  float sum = 0.0f, amax = 0.0f;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * step + tid;
    z[j] = 0.0f;
    if (e >= p.width) continue;
    float y = bf16_one(x[e]);
    if (kRes != 0) {
      y += load1<kRes == 0 ? 1 : kRes>(p.residual, base + e);
      store1<kRes == 0 ? 1 : kRes>(p.residual_out, base + e, y);
    }
    if (kW != 0) {
      sum = fmaf(y, y, sum);
      y *= load1<kW == 0 ? 1 : kW>(p.weight, e);
    }
    z[j] = y;
    amax = max_nan(amax, fabsf(y));
  }
  reduce_row(sum, amax, 0);
  const RowCodes codes(kW != 0, sum, amax, p.width, p.eps);
  if (tid == 0) p.scale[row] = codes.scale;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int e = j * step + tid;
    if (e < p.width) p.q[base + e] = (int8_t)(code_of(z[j] * codes.factor * codes.lift, codes.s, codes.r) & 0xFFu);
  }
}

// Rows wider than a CTA's registers hold: the row is read twice, an element
// at a time.  The first pass writes nothing, so the residual may be updated
// in place: each thread's second pass reads an element before it writes it.
template <int kRes, int kW>
__global__ void __launch_bounds__(kMaxRowThreads) long_rows_kernel(const RowParams p) {
  dev::griddep_launch_dependents();
  dev::griddep_wait();
  const int row = (int)blockIdx.x;
  const uint16_t* x = p.x + (long long)row * p.x_stride;
  const long long base = (long long)row * p.width;
  float sum = 0.0f, amax = 0.0f;
  for (int e = (int)threadIdx.x; e < p.width; e += (int)blockDim.x) {
    float y = bf16_one(x[e]);
    if (kRes != 0) y += load1<kRes == 0 ? 1 : kRes>(p.residual, base + e);
    if (kW != 0) {
      sum = fmaf(y, y, sum);
      y *= load1<kW == 0 ? 1 : kW>(p.weight, e);
    }
    amax = max_nan(amax, fabsf(y));
  }
  reduce_row(sum, amax, 0);
  const RowCodes codes(kW != 0, sum, amax, p.width, p.eps);
  if (threadIdx.x == 0) p.scale[row] = codes.scale;
  for (int e = (int)threadIdx.x; e < p.width; e += (int)blockDim.x) {
    float y = bf16_one(x[e]);
    if (kRes != 0) {
      y += load1<kRes == 0 ? 1 : kRes>(p.residual, base + e);
      store1<kRes == 0 ? 1 : kRes>(p.residual_out, base + e, y);
    }
    if (kW != 0) y *= load1<kW == 0 ? 1 : kW>(p.weight, e);
    p.q[base + e] = (int8_t)(code_of(y * codes.factor * codes.lift, codes.s, codes.r) & 0xFFu);
  }
}

template <int kRes, int kW>
cudaError_t launch_rows(const RowParams& p, bool wide, int num_sms, cudaStream_t stream) {
  const int vecs = (p.width + kVec - 1) / kVec;
  if (vecs > (wide ? 4 : 2) * kMaxRowThreads) {
    return launch_chained(long_rows_kernel<kRes, kW>, dim3((unsigned)p.rows), dim3(kMaxRowThreads), 0, 1, stream, p);
  }
  const auto threads = [&](int per) { return (unsigned)(((vecs + per - 1) / per + 31) & ~31); };
  if (!wide) {
    const dim3 grid((unsigned)p.rows);
    return vecs <= kMaxRowThreads
               ? launch_chained(odd_rows_kernel<kRes, kW, 8>, grid, dim3(threads(1)), 0, 1, stream, p)
               : launch_chained(odd_rows_kernel<kRes, kW, 16>, grid, dim3(threads(2)), 0, 1, stream, p);
  }
  // A warp a row of up to 512 features, four rows a CTA; else a CTA a row.  Few
  // rows get one vector a thread, for the shortest chain of latencies (one row
  // of 7168: 2.5 us, with four 3.3); many get two and a CTA takes several.
  const bool warp_rows = vecs <= 64;
  const bool few = p.rows <= 2 * num_sms;
  const int per = warp_rows ? (vecs <= 32 ? 1 : 2) : vecs > 2 * kMaxRowThreads ? 4 : few && vecs <= kMaxRowThreads ? 1 : 2;
  const dim3 block = warp_rows ? dim3(32, 4) : dim3(threads(per));
  // as many CTAs as are resident at once (64 registers a thread: 1024 threads an SM)
  const int resident = num_sms * (kMaxRowThreads / (int)(block.x * block.y));
  const int ctas = (p.rows + (int)block.y - 1) / (int)block.y;
  const dim3 grid((unsigned)(ctas < resident ? ctas : resident));
  if (per == 1) return launch_chained(rows_kernel<kRes, kW, 1>, grid, block, 0, 1, stream, p);
  if (per == 2) return launch_chained(rows_kernel<kRes, kW, 2>, grid, block, 0, 1, stream, p);
  return launch_chained(rows_kernel<kRes, kW, 4>, grid, block, 0, 1, stream, p);
}

template <int kRes>
cudaError_t launch_weight(const RowParams& p, int weight_type, bool wide, int num_sms, cudaStream_t stream) {
  if (weight_type == SPLITK_DTYPE_F32) return launch_rows<kRes, 2>(p, wide, num_sms, stream);
  return launch_rows<kRes, 1>(p, wide, num_sms, stream);
}

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1u)) == 0; }

// The checks both entry points share.
int check_rows(const void* x, long long x_stride, const void* q, const float* scale, int M, int D) {
  if (!x || !q || !scale) return SPLITK_ERR_NULL;
  if (M < 1 || D < 1 || x_stride < D || M > (1 << 30) || D > (1 << 30)) return SPLITK_ERR_INVALID_SHAPE;
  if (!aligned(x, 2) || !aligned(scale, 4)) return SPLITK_ERR_MISALIGNED;
  return SPLITK_OK;
}

}  // namespace

}  // namespace splitk

using namespace splitk;

extern "C" {

SPLITK_API int splitk_rmsnorm_i8(const void* x, long long x_stride, const void* residual, void* residual_out,
                                 int residual_type, const void* weight, int weight_type, float eps, void* q,
                                 float* scale, int M, int D, splitk_stream_t stream) {
  int rc = check_rows(x, x_stride, q, scale, M, D);
  if (rc != SPLITK_OK) return rc;
  if (!weight || (residual != nullptr) != (residual_out != nullptr)) return SPLITK_ERR_NULL;
  if (!(eps > 0.0f) || !(eps <= 3.4e38f)) return SPLITK_ERR_INVALID_ARGUMENT;
  if (weight_type != SPLITK_DTYPE_BF16 && weight_type != SPLITK_DTYPE_F32) return SPLITK_ERR_INVALID_ARGUMENT;
  if (residual && residual_type != SPLITK_DTYPE_BF16 && residual_type != SPLITK_DTYPE_F32) {
    return SPLITK_ERR_INVALID_ARGUMENT;
  }
  const uintptr_t r_size = residual_type == SPLITK_DTYPE_F32 ? 4u : 2u;
  const uintptr_t w_size = weight_type == SPLITK_DTYPE_F32 ? 4u : 2u;
  if (!aligned(weight, w_size)) return SPLITK_ERR_MISALIGNED;
  if (residual && (!aligned(residual, r_size) || !aligned(residual_out, r_size))) return SPLITK_ERR_MISALIGNED;
  DeviceSize dev;
  rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  const RowParams p{static_cast<const uint16_t*>(x), x_stride, residual, residual_out, weight, eps,
                    static_cast<int8_t*>(q), scale, M, D};
  const bool wide = D % kVec == 0 && x_stride % kVec == 0 && aligned(x, 16) && aligned(weight, 16) && aligned(q, 8) &&
                    aligned(residual, 16) && aligned(residual_out, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = !residual                               ? launch_weight<0>(p, weight_type, wide, dev.num_sms, s)
                        : residual_type == SPLITK_DTYPE_F32 ? launch_weight<2>(p, weight_type, wide, dev.num_sms, s)
                                                                : launch_weight<1>(p, weight_type, wide, dev.num_sms, s);
  return launched(e);
}

SPLITK_API int splitk_quantize_i8(const void* x, long long x_stride, void* q, float* scale, int M, int D,
                                  splitk_stream_t stream) {
  int rc = check_rows(x, x_stride, q, scale, M, D);
  if (rc != SPLITK_OK) return rc;
  DeviceSize dev;
  rc = require_device(&dev);
  if (rc != SPLITK_OK) return rc;
  const RowParams p{static_cast<const uint16_t*>(x), x_stride, nullptr, nullptr, nullptr, 0.0f,
                    static_cast<int8_t*>(q), scale, M, D};
  const bool wide = D % kVec == 0 && x_stride % kVec == 0 && aligned(x, 16) && aligned(q, 8);
  return launched(launch_rows<0, 0>(p, wide, dev.num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
