// The layer for few rows of X (1 to 32): W is read once and everything else is small,
// so what counts is how soon how much of W is under way.
//
// A workgroup takes 16 or 32 outputs (rows of W) and all rows of X; its KW wavefronts split the
// contraction and join their sums through LDS in a fixed order. A lane's 16-byte pieces of W go from
// memory to registers and into the matrix instruction as they are (lane l holds row l & 15, steps
// 8 (l >> 4) on), 4 or 8 pieces under way per lane; no LDS staging and no barrier before the end.
// Rows of X are padded to a multiple of 16 inside the instruction, whose work is hidden behind the
// loads; a row that does not exist is not loaded (a CU's address unit takes 64 bytes a cycle, and
// X would be half of them). Rows of any alignment are read as they are (memory takes unaligned
// accesses), so nothing is copied.
//
// Bound by the latency of a launch and one pass over W: bf16 1 x 4096 x 4096 takes 7.5 us (4.5 TB/s; a copy of
// 4 GiB reaches 4.7), fp16 13 x 2048 x 8192 8.1 us.
#include "linear_util.h"

namespace xtvxy {
namespace {

template <typename T>
struct Few {
  static constexpr int kChunk = 16 / sizeof(T);
  static constexpr int kSteps = 4 * kChunk;  // contraction steps of one piece per lane group
  typedef T piece __attribute__((ext_vector_type(kChunk)));
};

template <typename P>
__device__ __forceinline__ P load_piece(const void* p) {
  P v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

__device__ __forceinline__ f32x4 mfma_piece(f32x4 a, f32x4 b, f32x4 acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
  return acc;
}
__device__ __forceinline__ f32x4 mfma_piece(bf16x8 a, bf16x8 b, f32x4 acc) { return mfma_16x16(a, b, acc); }
__device__ __forceinline__ f32x4 mfma_piece(f16x8 a, f16x8 b, f32x4 acc) { return mfma_16x16(a, b, acc); }

// The piece's elements below `left`, the rest zero.
template <typename T, typename P>
__device__ __forceinline__ P load_part(const T* p, int64_t left) {
  P v = {};
#pragma unroll
  for (int i = 0; i < Few<T>::kChunk; ++i)
    if (i < left) v[i] = p[i];
  return v;
}

// MT tiles of 16 rows of X, NT of 16 outputs; KW wavefronts.
template <typename T, int MT, int NT, int KW>
__global__ __launch_bounds__(KW * 64) void product_few(ProductArgs a) {
  typedef typename Few<T>::piece piece;
  constexpr int kSteps = Few<T>::kSteps, kChunk = Few<T>::kChunk;
  constexpr int kAhead = MT * NT == 1 ? 8 : 4;
  __shared__ f32x4 sums[KW][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t j0 = (int64_t)blockIdx.x * 16 * NT;
  const int64_t k0 = ((int64_t)blockIdx.y * KW + wave) * a.k_per_split;
  const int64_t k1 = k0 + a.k_per_split < a.k ? k0 + a.k_per_split : a.k;
  const T* w[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    // an output that does not exist is formed as the last one and not stored
    const int64_t j = j0 + q * 16 + r < a.n ? j0 + q * 16 + r : a.n - 1;
    w[q] = static_cast<const T*>(a.B) + j * a.ldb + g * kChunk;
  }
  const T* x[MT];
  bool real[MT];  // a row of X that does not exist is zero and costs no load
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    real[t] = t * 16 + r < a.m;
    x[t] = static_cast<const T*>(a.A) + (real[t] ? t * 16 + r : 0) * a.lda + g * kChunk;
  }
  f32x4 acc[MT][NT] = {};
  int64_t k = k0;
  for (; k + kAhead * kSteps <= k1; k += kAhead * kSteps) {
    piece wp[kAhead][NT], xp[kAhead][MT] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int q = 0; q < NT; ++q) wp[u][q] = load_piece<piece>(w[q] + k + u * kSteps);
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if (real[t])
#pragma unroll
        for (int u = 0; u < kAhead; ++u) xp[u][t] = load_piece<piece>(x[t] + k + u * kSteps);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[t][q] = mfma_piece(wp[u][q], xp[u][t], acc[t][q]);
  }
  if (k < k1) {  // the rest in one go: its pieces, the very last one perhaps in part, are loaded together
    piece wp[kAhead][NT] = {}, xp[kAhead][MT] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t left = k1 - k - u * kSteps - g * kChunk;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        if (left >= kChunk) wp[u][q] = load_piece<piece>(w[q] + k + u * kSteps);
        else if (left > 0) wp[u][q] = load_part<T, piece>(w[q] + k + u * kSteps, left);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (!real[t]) continue;
        if (left >= kChunk) xp[u][t] = load_piece<piece>(x[t] + k + u * kSteps);
        else if (left > 0) xp[u][t] = load_part<T, piece>(x[t] + k + u * kSteps, left);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int q = 0; q < NT; ++q) acc[t][q] = mfma_piece(wp[u][q], xp[u][t], acc[t][q]);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int q = 0; q < NT; ++q) sums[wave][t * NT + q][lane] = acc[t][q];
  __syncthreads();
  for (int c = wave; c < MT * NT; c += KW) {
    f32x4 z = sums[0][c][lane];
    for (int s = 1; s < KW; ++s) z += sums[s][c][lane];
    const int64_t i = c / NT * 16 + r, j = j0 + c % NT * 16 + g * 4;
    if (i >= a.m || j >= a.n) continue;
    if (a.splits > 1 || a.in_parts)
      store4<float>(a.partial + ((int64_t)blockIdx.y * a.m + i) * a.n + j, z, a.n - j >= 4 ? 4 : (int)(a.n - j));
    else
      epilogue4<T>(a.e, i, j, a.n, z);
  }
}

template <typename T, int MT, int NT>
hipError_t few_waves(const ProductArgs& a, int waves, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 16 * NT - 1) / (16 * NT)), (unsigned)a.splits);
  if (waves == 8) product_few<T, MT, NT, 8><<<grid, 512, 0, s>>>(a);
  else product_few<T, MT, NT, 4><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t few_rows(const ProductArgs& a, int waves, int outputs, hipStream_t s) {
  if (a.m <= 16) return outputs == 32 ? few_waves<T, 1, 2>(a, waves, s) : few_waves<T, 1, 1>(a, waves, s);
  return outputs == 32 ? few_waves<T, 2, 2>(a, waves, s) : few_waves<T, 2, 1>(a, waves, s);
}

}  // namespace

hipError_t launch_product_few(const ProductArgs& a, int waves, int outputs, hipStream_t s) {
  if (a.type == kBf16) return few_rows<__bf16>(a, waves, outputs, s);
  if (a.type == kF16) return few_rows<_Float16>(a, waves, outputs, s);
  return few_rows<float>(a, waves, outputs, s);
}

}  // namespace xtvxy
