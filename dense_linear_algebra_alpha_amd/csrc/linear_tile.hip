// Products of any size, alignment, element type and operand order: 64 x 64 tiles, and the kernels
// around a product (the slope of the activation with its column sums, and the sum of a split
// contraction's parts).
#include "linear_util.h"

namespace xtvxy {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 256;
constexpr int kPitch = kTileDepth + 8;  // elements between tile rows in LDS: rows 16-byte aligned, banks spread

// One operand's 64 x 32 tile: rows r0.. of its kept index, steps k0.. of the contraction. A
// thread carries 8 neighbouring elements in registers from global memory to LDS; elements beyond
// `rows` or `k_end` are zero. In LDS the tile lies [row][step], whatever the order in memory.
template <typename T, bool kContractionMajor>
struct TileLoad {
  typename Vec<T>::x8 v;

  __device__ __forceinline__ void load(const T* base, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t k_end,
                                       bool wide) {
    const int t = threadIdx.x;
    const int64_t row = kContractionMajor ? r0 + (t & 7) * 8 : r0 + (t >> 2);
    const int64_t k = kContractionMajor ? k0 + (t >> 3) : k0 + (t & 3) * 8;
    const int64_t outer = kContractionMajor ? k : row, inner = kContractionMajor ? row : k;
    const int64_t outer_end = kContractionMajor ? k_end : rows, inner_end = kContractionMajor ? rows : k_end;
    const int64_t left = outer < outer_end ? inner_end - inner : 0;
    const T* p = base + outer * ld + inner;
    if (wide && left >= 8) {
      v = *reinterpret_cast<const typename Vec<T>::x8*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : (T)0.0f;
    }
  }

  __device__ __forceinline__ void store(T* lds) const {
    const int t = threadIdx.x;
    if (kContractionMajor) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lds[((t & 7) * 8 + i) * kPitch + (t >> 3)] = v[i];
    } else {
      *reinterpret_cast<typename Vec<T>::x8*>(lds + (t >> 2) * kPitch + (t & 3) * 8) = v;
    }
  }
};

// One 64 x 64 tile of C per workgroup, four wavefronts of 32 x 32 each. The product is formed
// transposed (B's rows as the matrix instruction's first operand), so that a lane ends with four
// neighbouring columns of one row of C. The next step's elements are in flight while the present
// one's products run.
template <typename T, bool kAMajor, bool kBMajor>
__global__ __launch_bounds__(kThreads) void product_tile(ProductArgs a) {
  __shared__ __align__(16) T sa[kTile * kPitch], sb[kTile * kPitch];
  typedef typename Vec<T>::x8 frag;
  const int64_t tiles_n = (a.n + kTile - 1) / kTile;
  const int64_t i0 = (blockIdx.x / tiles_n) * kTile, j0 = (blockIdx.x % tiles_n) * kTile;
  const int64_t k0 = (int64_t)blockIdx.y * a.k_per_split;
  const int64_t k_end = k0 + a.k_per_split < a.k ? k0 + a.k_per_split : a.k;
  const T* A = static_cast<const T*>(a.A);
  const T* B = static_cast<const T*>(a.B);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
  const int r = lane & 15, g = lane >> 4;

  f32x4 acc[2][2] = {};
  TileLoad<T, kAMajor> la;
  TileLoad<T, kBMajor> lb;
  la.load(A, a.lda, i0, a.m, k0, k_end, a.a_wide);
  lb.load(B, a.ldb, j0, a.n, k0, k_end, a.b_wide);
  for (int64_t k = k0; k < k_end; k += kTileDepth) {
    la.store(sa);
    lb.store(sb);
    __syncthreads();
    if (k + kTileDepth < k_end) {
      la.load(A, a.lda, i0, a.m, k + kTileDepth, k_end, a.a_wide);
      lb.load(B, a.ldb, j0, a.n, k + kTileDepth, k_end, a.b_wide);
    }
    frag fa[2], fb[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      fa[x] = *reinterpret_cast<const frag*>(sa + (wi + x * 16 + r) * kPitch + g * 8);
      fb[x] = *reinterpret_cast<const frag*>(sb + (wj + x * 16 + r) * kPitch + g * 8);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) acc[x][y] = mfma_16x16(fb[y], fa[x], acc[x][y]);
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int64_t i = i0 + wi + x * 16 + r, j = j0 + wj + y * 16 + g * 4;
      if (i >= a.m || j >= a.n) continue;
      if (a.splits > 1) {
        float* p = a.partial + ((int64_t)blockIdx.y * a.m + i) * a.n + j;
        store4<float>(p, acc[x][y], a.n - j >= 4 ? 4 : (int)(a.n - j), a.n % 4 == 0);
      } else {
        epilogue4<T>(a.e, i, j, a.n, acc[x][y]);
      }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void product_finish(ProductArgs a) {
  const int64_t quads = (a.n + 3) / 4, q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (q >= a.m * quads) return;
  const int64_t i = q / quads, j = (q % quads) * 4;
  const int count = a.n - j >= 4 ? 4 : (int)(a.n - j);
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.splits; ++s) z += load4<float>(a.partial + ((int64_t)s * a.m + i) * a.n + j, count, a.n % 4 == 0);
  epilogue4<T>(a.e, i, j, a.n, z);
}

// d = g act'(pre) in fp32, stored in the element type; the column sums db take d before that
// rounding. A workgroup walks rows_per_group rows; a thread owns 8 neighbouring columns.
template <typename T, int kAct>
__global__ __launch_bounds__(kThreads) void slope_rows(SlopeArgs a) {
  const int64_t j = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
  const int part = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_group;
  const int64_t r1 = r0 + a.rows_per_group < a.m ? r0 + a.rows_per_group : a.m;
  const T* G = static_cast<const T*>(a.g);
  const T* P = static_cast<const T*>(a.pre);
  T* D = static_cast<T*>(a.d);
  typedef typename Vec<T>::x8 v8;
  float sum[8] = {};
  const int count = a.n - j >= 8 ? 8 : (a.n > j ? (int)(a.n - j) : 0);
  if (count > 0) {
    for (int64_t i = r0 + part; i < r1; i += kThreads / 64) {
      float x[8];
      if (a.wide && count == 8) {
        const v8 g = *reinterpret_cast<const v8*>(G + i * a.ldg + j);
        v8 z = g, o;
        if (kAct != XTVXY_ACT_NONE) z = *reinterpret_cast<const v8*>(P + i * a.ldp + j);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          x[c] = (float)g[c];
          if (kAct != XTVXY_ACT_NONE) x[c] *= slope<kAct>((float)z[c]);
          o[c] = (T)x[c];
        }
        if (D) *reinterpret_cast<v8*>(D + i * a.ldd + j) = o;
      } else {
        v8 o = {};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          x[c] = 0.0f;
          if (c < count) {
            x[c] = (float)G[i * a.ldg + j + c];
            if (kAct != XTVXY_ACT_NONE) x[c] *= slope<kAct>((float)P[i * a.ldp + j + c]);
            o[c] = (T)x[c];
          }
        }
        if (D) *reinterpret_cast<v8*>(D + i * a.ldd + j) = o;  // ldd is a multiple of 8
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += x[c];
    }
  }
  if (!a.sums) return;
  __shared__ float part_sums[kThreads / 64 - 1][64][9];
  if (part > 0) {
#pragma unroll
    for (int c = 0; c < 8; ++c) part_sums[part - 1][threadIdx.x & 63][c] = sum[c];
  }
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      for (int p = 0; p < kThreads / 64 - 1; ++p) sum[c] += part_sums[p][threadIdx.x][c];
      if (c < count) a.sums[(int64_t)blockIdx.y * a.n + j + c] = sum[c];
    }
  }
}

// 16 bytes of a row at a time; the source may have any alignment (memory takes unaligned accesses).
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_rows(PackArgs a) {
  constexpr int kChunk = 16 / sizeof(T);
  typedef T chunk __attribute__((ext_vector_type(kChunk)));
  const PackJob& job = a.job[blockIdx.y];
  const int64_t chunks = job.ldd / kChunk, total = job.rows * chunks;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < total; at += (int64_t)gridDim.x * kThreads) {
    const int64_t i = at / chunks, c = (at % chunks) * kChunk;
    const T* p = static_cast<const T*>(job.src) + i * job.ld + c;
    chunk v = {};
    if (job.cols - c >= kChunk) {
      __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
      for (int x = 0; x < kChunk; ++x)
        if (c + x < job.cols) v[x] = p[x];
    }
    *reinterpret_cast<chunk*>(static_cast<T*>(job.dst) + i * job.ldd + c) = v;
  }
}

__global__ __launch_bounds__(kThreads) void column_finish(const float* sums, int64_t groups, int64_t n, float* db) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= n) return;
  double s = 0.0;
  for (int64_t g = 0; g < groups; ++g) s += (double)sums[g * n + j];
  db[j] = (float)s;
}

template <typename T>
hipError_t tile_for(const ProductArgs& a, hipStream_t s) {
  const int64_t tiles = ((a.m + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile);
  const dim3 grid((unsigned)tiles, (unsigned)a.splits);
  if (a.a_contraction_major && a.b_contraction_major)
    product_tile<T, true, true><<<grid, kThreads, 0, s>>>(a);
  else if (a.b_contraction_major)
    product_tile<T, false, true><<<grid, kThreads, 0, s>>>(a);
  else
    product_tile<T, false, false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t slope_for(const SlopeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 511) / 512), (unsigned)a.groups);
  switch (a.pre ? a.act : XTVXY_ACT_NONE) {
    case XTVXY_ACT_RELU: slope_rows<T, XTVXY_ACT_RELU><<<grid, kThreads, 0, s>>>(a); break;
    case XTVXY_ACT_GELU: slope_rows<T, XTVXY_ACT_GELU><<<grid, kThreads, 0, s>>>(a); break;
    case XTVXY_ACT_GELU_TANH: slope_rows<T, XTVXY_ACT_GELU_TANH><<<grid, kThreads, 0, s>>>(a); break;
    case XTVXY_ACT_SILU: slope_rows<T, XTVXY_ACT_SILU><<<grid, kThreads, 0, s>>>(a); break;
    default: slope_rows<T, XTVXY_ACT_NONE><<<grid, kThreads, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_tile(const ProductArgs& a, hipStream_t s) {
  if (a.type == kBf16) return tile_for<__bf16>(a, s);
  if (a.type == kF16) return tile_for<_Float16>(a, s);
  return tile_for<float>(a, s);
}

hipError_t launch_product_finish(const ProductArgs& a, hipStream_t s) {
  const int64_t quads = a.m * ((a.n + 3) / 4);
  const unsigned grid = (unsigned)((quads + kThreads - 1) / kThreads);
  if (a.type == kBf16) product_finish<__bf16><<<grid, kThreads, 0, s>>>(a);
  else if (a.type == kF16) product_finish<_Float16><<<grid, kThreads, 0, s>>>(a);
  else product_finish<float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_slope(const SlopeArgs& a, hipStream_t s) {
  if (a.type == kBf16) return slope_for<__bf16>(a, s);
  if (a.type == kF16) return slope_for<_Float16>(a, s);
  return slope_for<float>(a, s);
}

hipError_t launch_pack(const PackArgs& a, int type, hipStream_t s) {
  int64_t most = 1;
  for (int j = 0; j < a.jobs; ++j) {
    const int64_t groups = (a.job[j].rows * (a.job[j].ldd * elem_size(type) / 16) + kThreads - 1) / kThreads;
    most = groups > most ? groups : most;
  }
  const dim3 grid((unsigned)(most < 8192 ? most : 8192), (unsigned)a.jobs);
  if (type == kF32) pack_rows<float><<<grid, kThreads, 0, s>>>(a);
  else pack_rows<_Float16><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_column_finish(const float* sums, int64_t groups, int64_t n, float* db, hipStream_t s) {
  column_finish<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(sums, groups, n, db);
  return hipGetLastError();
}

}  // namespace xtvxy
