// Device helpers of the fully connected layer: element types, activations and their slopes, and
// the epilogue that the product kernels share.
#pragma once

#include "device_util.h"
#include "linear.h"

namespace xtvxy {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  typedef f32x4 x4;
  typedef f32x8 x8;
};
template <>
struct Vec<__bf16> {
  typedef bf16x4 x4;
  typedef bf16x8 x8;
};
template <>
struct Vec<_Float16> {
  typedef f16x4 x4;
  typedef f16x8 x8;
};

// acc += sum over 32 contraction steps for a 16 x 16 tile. Lane l brings the 8 steps of row
// l & 15 that belong to group l >> 4, the same steps for a and b; it gets column l & 15 of rows
// 4 (l >> 4) + 0..3 of a's index by b's.
__device__ __forceinline__ f32x4 mfma_16x16(bf16x8 a, bf16x8 b, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_16x16(f16x8 a, f16x8 b, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
}
// fp32: eight products of 4 steps each; step s takes element s of each group's eight.
__device__ __forceinline__ f32x4 mfma_16x16(f32x8 a, f32x8 b, f32x4 acc) {
#pragma unroll
  for (int s = 0; s < 8; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
  return acc;
}

// exp(x) = 2^(x log2 e) by the hardware's exponential (1 unit in the last place). The product's
// rounding costs |x| 2^-24 relative to the result, which is itself small where |x| is large.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// Phi(z) = erfc(-z / sqrt 2) / 2, the normal distribution function; *density gets exp(-z^2 / 2).
// erfc(a) = exp(-a^2) P(1 / (1 + c a)), a >= 0 (Hastings' form; Abramowitz and Stegun, 7.1.26, has coefficients
// for the absolute error), P fitted here to the least largest relative error: degree 9
// for fp32 results and for slopes (whose sums db are fp32), 4.2e-8 on [0, 14], 2.9e-7 as evaluated;
// degree 5 for 16-bit results, 2.2e-5 (half a step of fp16 is 2.4e-4). One reciprocal, one exponential
// and 6 or 10 fused multiply-adds; the library's erfcf takes about 40 operations.
template <bool kFast>
__device__ __forceinline__ float normal_cdf(float z, float* density) {
  const float x = fast_exp(-0.5f * z * z);
  float p;
  if (kFast) {
    const float t = fast_rcp(fmaf(fabsf(z), 0.35f * 0.70710678f, 1.0f));
    p = 0.5491096602476102f;
    p = fmaf(p, t, -0.34366955118616876f);
    p = fmaf(p, t, 0.474523528705992f);
    p = fmaf(p, t, 0.1100193553124311f);
    p = fmaf(p, t, 0.2108346123613167f);
    p = fmaf(p, t, -0.0008098688139377294f);
  } else {
    const float t = fast_rcp(fmaf(fabsf(z), 0.5f * 0.70710678f, 1.0f));
    p = -0.058820225176986256f;
    p = fmaf(p, t, 0.2832750472588048f);
    p = fmaf(p, t, -0.48426956863631826f);
    p = fmaf(p, t, 0.2743361059568525f);
    p = fmaf(p, t, -0.02367546535291248f);
    p = fmaf(p, t, 0.20118783384543076f);
    p = fmaf(p, t, 0.24359225429523224f);
    p = fmaf(p, t, 0.28227702194312615f);
    p = fmaf(p, t, 0.2820974844117237f);
    p = fmaf(p, t, -5.308339471779765e-07f);
  }
  const float tail = 0.5f * p * x;  // Phi(-|z|)
  *density = x;
  return z < 0.0f ? tail : 1.0f - tail;
}

// Twice the argument of the tanh in gelu's tanh form: (1 + tanh u) / 2 = 1 / (1 + exp(-2u)).
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return z * fmaf(z * z, 2.0f * 0.79788456f * 0.044715f, 2.0f * 0.79788456f);
}

__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

template <bool kFast, int kAct>
__device__ __forceinline__ float activation(float z) {
  if (kAct == XTVXY_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays
  if (kAct == XTVXY_ACT_GELU) {
    float x;
    return z * normal_cdf<kFast>(z, &x);
  }
  if (kAct == XTVXY_ACT_GELU_TANH) return z * sigmoid(gelu_tanh_arg(z));
  if (kAct == XTVXY_ACT_SILU) return z * sigmoid(z);
  return z;
}

// d activation / dz.
template <int kAct>
__device__ __forceinline__ float slope(float z) {
  if (kAct == XTVXY_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (kAct == XTVXY_ACT_GELU) {
    float x;
    const float c = normal_cdf<false>(z, &x);
    return fmaf(z * x, 0.39894228f, c);
  }
  if (kAct == XTVXY_ACT_GELU_TANH) {
    const float q = sigmoid(gelu_tanh_arg(z));
    const float w = q * (1.0f - q);
    // where the sigmoid is flat its slope is zero whatever z^3 has grown to
    return w == 0.0f ? q : fmaf(z * w, fmaf(z * z, 6.0f * 0.79788456f * 0.044715f, 2.0f * 0.79788456f), q);
  }
  if (kAct == XTVXY_ACT_SILU) {
    const float q = sigmoid(z);
    return q * fmaf(z, 1.0f - q, 1.0f);
  }
  return 1.0f;
}

// N = 4 or 8 elements of a row of which the first `count` exist (the rest come out as zero). Memory takes
// vector accesses of any alignment, so only a row's last elements go piecewise, in at most three accesses:
// with one access per element the ends of rows of odd length cost more than the rest of the epilogue.
template <typename T, int N>
__device__ __forceinline__ void load_elems(const T* p, int count, T (&x)[N]) {
  if (count >= N) {
    __builtin_memcpy(x, p, sizeof(T) * N);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = (T)0.0f;
  T four[4] = {}, two[2] = {}, one = (T)0.0f;
  if (N == 8 && (count & 4)) __builtin_memcpy(four, p, sizeof(four));
  const T* q = p + (count & (N == 8 ? 4 : 0));
  if (count & 2) __builtin_memcpy(two, q, sizeof(two));
  if (count & 1) one = q[count & 2];
  const int at = N == 8 ? count & 4 : 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (N == 8 && i < 4 && at) x[i] = four[i];
    if (i >= at && i < at + 2 && (count & 2)) x[i] = two[(i - at) & 1];
    if ((count & 1) && i == count - 1) x[i] = one;
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_elems(T* p, int count, const T (&x)[N]) {
  if (count >= N) {
    __builtin_memcpy(p, x, sizeof(T) * N);
    return;
  }
  T* q = p;
  T y[4] = {x[0], x[1], x[2], x[3]};
  if (N == 8 && (count & 4)) {
    __builtin_memcpy(q, y, sizeof(y));
    q += 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = x[(i + 4) % N];
  }
  T z = y[0];
  if (count & 2) {
    __builtin_memcpy(q, y, 2 * sizeof(T));
    q += 2;
    z = y[2];
  }
  if (count & 1) *q = z;
}

template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p, int count) {
  T x[4];
  load_elems<T, 4>(p, count, x);
  return {(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}

template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 v, int count) {
  const T x[4] = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  store_elems<T, 4>(p, count, x);
}

template <bool kFast>
__device__ __forceinline__ f32x4 activation4(f32x4 z, int act) {
  f32x4 r = z;
  switch (act) {
#define XTVXY_ACT_CASE(A)                                                  \
  case A:                                                                  \
    _Pragma("unroll") for (int i = 0; i < 4; ++i) r[i] = activation<kFast, A>(z[i]); \
    break;
    XTVXY_ACT_CASE(XTVXY_ACT_RELU)
    XTVXY_ACT_CASE(XTVXY_ACT_GELU)
    XTVXY_ACT_CASE(XTVXY_ACT_GELU_TANH)
    XTVXY_ACT_CASE(XTVXY_ACT_SILU)
#undef XTVXY_ACT_CASE
    default: break;
  }
  return r;
}

// The epilogue of four neighbouring columns j..j+3 of row i; columns >= n do not exist. z is kept
// in fp32 through bias, activation and residual and rounded once per stored element.
template <typename T>
__device__ __forceinline__ void epilogue4(const LinearEpilogue& e, int64_t i, int64_t j, int64_t n, f32x4 z) {
  const int count = n - j >= 4 ? 4 : (int)(n - j);
  if (count <= 0) return;
  if (e.bias) z += load4<float>(e.bias + j, count);
  if (e.pre) store4<T>(static_cast<T*>(e.pre) + i * e.ldp + j, z, count);
  f32x4 y = activation4<sizeof(T) == 2>(z, e.act);
  if (e.residual) y += load4<T>(static_cast<const T*>(e.residual) + i * e.ldr + j, count);
  store4<T>(static_cast<T*>(e.out) + i * e.ldo + j, y, count);
}

// Place of the t-th tile of a product: tiles are ordered in bands of kBand tile rows, so that
// neighbours in the order share operands.
__device__ __forceinline__ void tile_of(const ProductArgs& a, uint32_t t, int64_t* tm, int64_t* tn) {
  constexpr uint32_t kBand = 4;
  const uint32_t tiles_m = (uint32_t)((a.m + a.tile - 1) / a.tile), tiles_n = (uint32_t)((a.n + a.tile - 1) / a.tile);
  const uint32_t band_tiles = kBand * tiles_n, band = t / band_tiles, in = t % band_tiles;
  const uint32_t rows = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  *tm = band * kBand + in % rows;
  *tn = in / rows;
}

// Workgroups go to the 8 XCDs in turn, each of which has an L2 of its own: of `count` positions, workgroup
// id takes one of its XCD's contiguous range.
__device__ __forceinline__ uint32_t spread(uint32_t id, uint32_t count) {
  constexpr uint32_t kXcds = 8;
  const uint32_t x = id % kXcds, q = count / kXcds, r = count % kXcds;
  return x * q + (x < r ? x : r) + id / kXcds;
}

// db[j] = the sum of sums[.][n] over its rows for the 16 columns of workgroup `group` (256 threads): a
// thread adds every 16th row of a column, the 16 partial sums join in LDS (2 KiB), in fp64 and in a
// fixed order. 16 loads of a column are under way at once; one thread per column would wait for each.
constexpr int kSumColumns = 16;
__device__ __forceinline__ void column_sum(const float* sums, int64_t rows, int64_t n, float* db, int64_t group, double* lds) {
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int64_t j = group * kSumColumns + c;
  double s = 0.0;
  if (j < n) {
#pragma unroll 4
    for (int64_t g = slot; g < rows; g += 16) s += (double)sums[g * n + j];
  }
  lds[slot * 16 + c] = s;
  __syncthreads();
  if (slot == 0 && j < n) {
    for (int p = 1; p < 16; ++p) s += lds[p * 16 + c];
    db[j] = (float)s;
  }
}

}  // namespace xtvxy
