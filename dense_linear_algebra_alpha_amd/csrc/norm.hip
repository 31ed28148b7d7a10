// Layer norm over the rows of a matrix, and its gradient.
//
//     mean_i = sum_j x_ij / n,  rstd_i = 1 / sqrt(sum_j (x_ij - mean_i)^2 / n + eps),  xhat = (x - mean) rstd,
//     out = xhat weight + bias;
//     h = g weight,  dX = rstd (h - sum_j h_ij / n - xhat sum_j h_ij xhat_ij / n),
//     dweight = sum_i g_ij xhat_ij,  dbias = sum_i g_ij.
//
// Both are bound by memory: the forward pass reads and writes each element once, the gradient reads two and
// writes one. Forward: a row is shared by 16, 64, 256 or 1024 threads, in whose registers it stays between its sums and its
// output; threads keep their columns from row to row, so weight and bias are loaded once per workgroup, and the next row is
// loaded before the sums of the current one are joined. (In 16 bits, rows of more than 16384 columns are more than the
// registers hold: 75 of a thread's go to scratch memory.) Gradient: a row is shared by 16 to 1024 threads, every power of
// two; its column sums stay in registers, the weight is reloaded for every row, and the next row is loaded ahead but for fp32
// rows of more than 8192 columns. Rows shorter than 16 bytes, or longer than the registers, have kernels of their own.
//
// us of the kernels: forward with statistics, bf16 16384 x 4096, alone 53 (5.1 TB/s, what a copy reaches), one of many 47;
// 1 x 4096 2.3; gradient of the same 78 (5.3 TB/s) and 5 for the columns' sums of 256 workgroups, fp32 5001 x 1111 16 and 4.
//
// A row's last chunk of 16 bytes, where n is no multiple of one, is the last 16 bytes of the row: memory
// takes any alignment, a branch around its loads would make every row wait for them. What it shares with
// the chunk before counts once in the sums and is stored twice with the same value.
#include <type_traits>

#include "linear_util.h"
#include "norm.h"

namespace xtvxy {
namespace {

template <typename T>
constexpr int kChunkOf = 16 / sizeof(T);  // elements of a chunk

typedef u32x4 unaligned_chunk __attribute__((aligned(2)));
constexpr int64_t kL2Bytes = 32 << 20;  // of the eight XCDs

// kStreamed: past the L2s, for outputs that do not fit there.
template <bool kStreamed, typename T, int V>
__device__ __forceinline__ void store_chunk(T* p, const T (&o)[V]) {
  u32x4 v;
  __builtin_memcpy(&v, o, 16);
  if (kStreamed) __builtin_nontemporal_store(v, reinterpret_cast<unaligned_chunk*>(p));
  else __builtin_memcpy(p, &v, 16);
}

// The chunks of a row that a thread owns: chunk c begins at column at[c]; the first skip[c] of its elements
// belong to another chunk (all of them where the chunk is beyond the row).
template <typename T, int L, int C>
struct Columns {
  static constexpr int V = kChunkOf<T>;
  int32_t at[C], skip[C];
  __device__ __forceinline__ Columns(int64_t n, int t) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t j = (int64_t)(c * L + t) * V, last = n - V;
      at[c] = (int32_t)(j < last ? j : last);
      skip[c] = j < last ? 0 : j - last < V ? (int32_t)(j - last) : V;
    }
  }
};

template <typename T, int C>
struct Chunks {
  static constexpr int V = kChunkOf<T>;
  T e[C][V];
  template <typename K>
  __device__ __forceinline__ void load(const T* row, const K& k) {
#pragma unroll
    for (int c = 0; c < C; ++c) __builtin_memcpy(e[c], row + k.at[c], 16);
  }
};

template <int V, typename K, int C>
__device__ __forceinline__ void load_vector(const float* p, const K& k, float otherwise, float (&v)[C][V]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (p) {
      __builtin_memcpy(v[c], p + k.at[c], 4 * V);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[c][e] = otherwise;
    }
  }
}

// x over the wavefronts of a row (waves of them, slots of `lds` from `first` on), in a fixed order.
template <int kWaves>
__device__ __forceinline__ float row_sum(const float* lds, int first) {
  float s = lds[first];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += lds[first + w];
  return s;
}

// A row's squares may have left fp32 where its variance (with eps) is infinite or NaN (distances beyond 1.8e19), or below 2^-100
// (next to an eps as small, below 1e-19).
constexpr float kLeastVariance = 0x1p-100f, kMostRstd = 0x1p50f;
__device__ __forceinline__ bool out_of_range(float variance) { return !(variance >= kLeastVariance && variance < __builtin_inff()); }

// The sum over a workgroup of kThreads, or over a wavefront (64), the same in every thread; `lds` has kThreads / 64 doubles.
template <int kThreads>
__device__ __forceinline__ double wide_sum(double x, double* lds) {
#pragma unroll
  for (int by = 1; by < 64; by *= 2) x += __shfl_xor(x, by);
  if constexpr (kThreads > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
    for (int w = 1; w < kThreads / 64; ++w) x += lds[w];
  }
  return x;
}

// Row i, by thread t of kThreads, with its sums in fp64; where not `always`, only if its variance is below kLeastVariance.
template <typename T, int kThreads>
__device__ __forceinline__ void wide_row(const NormArgs& a, int64_t i, int t, double* lds, bool always) {
  const T* x = static_cast<const T*>(a.x) + i * a.ldx;
  T* out = static_cast<T*>(a.out) + i * a.ldo;
  double s = 0.0, q = 0.0;
  for (int64_t j = t; j < a.n; j += kThreads) s += (double)(float)x[j];
  const float mean = (float)(wide_sum<kThreads>(s, lds) / (double)a.n);
  for (int64_t j = t; j < a.n; j += kThreads) {
    const double d = (double)((float)x[j] - mean);
    q += d * d;
  }
  const double variance = wide_sum<kThreads>(q, lds) / (double)a.n + (double)a.eps;
  if (!always && variance >= kLeastVariance) return;
  const float rstd = (float)(1.0 / sqrt(variance));
  if (t == 0) {
    if (a.mean) a.mean[i] = mean;
    if (a.rstd) a.rstd[i] = rstd;
  }
  for (int64_t j = t; j < a.n; j += kThreads)
    out[j] = (T)fmaf(((float)x[j] - mean) * rstd, a.weight ? a.weight[j] : 1.0f, a.bias ? a.bias[j] : 0.0f);
}

// A row's mean and sum of squared distances from it. Each wavefront forms its own mean first and takes
// distances from that (no cancellation); the wavefronts' (mean, distances) join as
//     mean = sum n_w mean_w / n,  sum = sum_w (sum_w + n_w (mean_w - mean)^2).
template <typename T, int L, int C, bool kStreamed>
__global__ __launch_bounds__(L < 256 ? 256 : L) void norm_rows(NormArgs a) {
  constexpr int V = kChunkOf<T>, kBlock = L < 256 ? 256 : L, kRows = kBlock / L, kWaves = L / 64, kGroup = L < 64 ? L : 64;
  __shared__ float part[2][2][kBlock / 64];
  __shared__ double wide[kBlock / 64];
  const int t = threadIdx.x % L, sub = threadIdx.x / L, lane = threadIdx.x & 63;
  const Columns<T, L, C> k(a.n, t);
  float w[C][V], b[C][V];
  load_vector<V>(a.weight, k, 1.0f, w);
  load_vector<V>(a.bias, k, 0.0f, b);
  const float n = (float)a.n;
  int own = 0;  // elements of the row that this thread counts
#pragma unroll
  for (int c = 0; c < C; ++c) own += V - k.skip[c];
  const float mine = group_sum((float)own, kGroup);
  float counts[kWaves > 0 ? kWaves : 1];  // of each wavefront of the row
  if constexpr (kWaves > 1) {
    if (lane == 0) part[0][0][threadIdx.x / 64] = mine;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kWaves; ++v) counts[v] = part[0][0][sub * kWaves + v];
    __syncthreads();
  }
  const T* X = static_cast<const T*>(a.x);
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t i = (int64_t)blockIdx.x * kRows + sub;
  Chunks<T, C> next;
  next.load(X + (i < a.m ? i : a.m - 1) * a.ldx, k);
  int turn = 0;
  uint32_t largest = 0;  // rstd, as bits: NaN is beyond all
  for (int64_t i0 = (int64_t)blockIdx.x * kRows; i0 < a.m; i0 += step, i += step, turn ^= 1) {
    float x[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) x[c][e] = (float)next.e[c][e];
    if (i0 + step < a.m) next.load(X + (i + step < a.m ? i + step : a.m - 1) * a.ldx, k);
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) s += e >= k.skip[c] ? x[c][e] : 0.0f;
    // divided: the mean of a constant row is that constant
    float mean = mine > 0.0f ? group_sum(s, kGroup) / mine : 0.0f, q = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = x[c][e] - mean;
        q += e >= k.skip[c] ? d * d : 0.0f;
      }
    q = group_sum(q, kGroup);
    if constexpr (kWaves > 1) {
      if (lane == 0) {
        part[turn][0][threadIdx.x / 64] = mean;
        part[turn][1][threadIdx.x / 64] = q;
      }
      __syncthreads();
      const float* means = &part[turn][0][sub * kWaves];
      const float* squares = &part[turn][1][sub * kWaves];
      float total = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) total += counts[v] * means[v];
      mean = total / n;
      q = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const float d = means[v] - mean;
        q += squares[v] + counts[v] * d * d;
      }
    }
    if (i >= a.m) continue;
    const float variance = q / n + a.eps;
    const float rstd = fmaf(variance, 0.0f, 1.0f / sqrtf(variance));  // NaN of an infinite variance
    const uint32_t bits = __float_as_uint(rstd);
    largest = largest > bits ? largest : bits;
    if (t == 0) {
      if (a.mean) a.mean[i] = mean;
      if (a.rstd) a.rstd[i] = rstd;
    }
    T* out = static_cast<T*>(a.out) + i * a.ldo;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (k.skip[c] == V) continue;
      T o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = (T)fmaf((x[c][e] - mean) * rstd, w[c][e], b[c][e]);
      store_chunk<kStreamed>(out + k.at[c], o);
    }
  }
  // Rows out of range (of an infinite variance all outputs are NaN so far) once more, by the workgroup or, where a wavefront
  // has rows of its own, by it. (us, 10392 x 1269 of bf16 13.50, without the two operations a row that look for them 13.49,
  // handled where they occur 13.9; 5001 x 1111 of fp32 12.9, 12.7; 2000 x 32768 of bf16 121, 117.)
  constexpr int kTeam = L > 64 ? kBlock : 64, kTeamRows = kTeam / L;
  if (!__any(largest > __float_as_uint(kMostRstd))) return;  // alike in a whole team
  __threadfence();
  if (L > 64) __syncthreads();
  for (int64_t i0 = (int64_t)blockIdx.x * kRows + threadIdx.x / kTeam * kTeamRows; i0 < a.m; i0 += step)
    for (int64_t row = i0; row < i0 + kTeamRows && row < a.m; ++row) {
      const float first = (float)static_cast<const T*>(a.out)[row * a.ldo];
      wide_row<T, kTeam>(a, row, threadIdx.x % kTeam, wide, first != first);
    }
}

// Rows longer than the registers of 1024 threads: a workgroup walks the row once for the mean, once for the distances and
// once for the output (the second and third time out of L2). The sums are fp64: a thread's may have 2^17 terms. In fp32 the
// mean of 4 10^7 times 1.1 drifts to 1.1002, which 1 / sqrt(eps) makes 0.06. (us, fp32: 2000 x 20001 111, summed in fp32 104;
// 1000 x 100003 385, 375.)
template <typename T>
__global__ __launch_bounds__(1024) void norm_long(NormArgs a) {
  __shared__ double lds[1024 / 64];
  for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) wide_row<T, 1024>(a, i, threadIdx.x, lds, true);
}

// Rows shorter than a chunk, a wavefront each.
template <typename T>
__global__ __launch_bounds__(64) void norm_short(NormArgs a) {
  const int j = threadIdx.x;
  const bool on = j < a.n;
  for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) {
    const float x = on ? (float)static_cast<const T*>(a.x)[i * a.ldx + j] : 0.0f;
    const float mean = group_sum(x, 64) / (float)a.n, d = on ? x - mean : 0.0f;
    const float variance = group_sum(d * d, 64) / (float)a.n + a.eps, rstd = 1.0f / sqrtf(variance);
    if (out_of_range(variance)) {
      wide_row<T, 64>(a, i, threadIdx.x, nullptr, true);
      continue;
    }
    if (j == 0) {
      if (a.mean) a.mean[i] = mean;
      if (a.rstd) a.rstd[i] = rstd;
    }
    if (on) static_cast<T*>(a.out)[i * a.ldo + j] = (T)fmaf(d * rstd, a.weight ? a.weight[j] : 1.0f, a.bias ? a.bias[j] : 0.0f);
  }
}

// ---------------------------------------------------------------------------
// the gradient
// ---------------------------------------------------------------------------

constexpr int kGradientThreads = 1024;

// A workgroup takes 1024 / L rows at a time. Its rows' column sums join in LDS at the end.
template <typename T, int L, int C>
__global__ __launch_bounds__(kGradientThreads) void norm_gradient_rows(NormGradientArgs a) {
  constexpr int V = kChunkOf<T>, kRows = kGradientThreads / L, kWaves = L / 64, kGroup = L < 64 ? L : 64;
  __shared__ float part[2][2][kGradientThreads / 64];
  __shared__ __align__(16) float join[kRows][L * V];
  const int t = threadIdx.x % L, sub = threadIdx.x / L, lane = threadIdx.x & 63;
  const Columns<T, L, C> k(a.n, t);
  float dw[C][V] = {}, db[C][V] = {};
  const float inv_n = 1.0f / (float)a.n;
  const T* X = static_cast<const T*>(a.x);
  const T* G = static_cast<const T*>(a.g);
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t i = (int64_t)blockIdx.x * kRows + sub;
  Chunks<T, C> x, g;
  float mean = 0.0f, rstd = 0.0f;
  const auto load = [&](int64_t row) {
    row = row < a.m ? row : a.m - 1;
    x.load(X + row * a.ldx, k);
    g.load(G + row * a.ldg, k);
    mean = a.mean[row];
    rstd = a.rstd[row];
  };
  constexpr bool kAhead = C * V < 16 || sizeof(T) == 2;
  if (kAhead) load(i);
  int turn = 0;
  for (int64_t i0 = (int64_t)blockIdx.x * kRows; i0 < a.m; i0 += step, i += step, turn ^= 1) {
    if (!kAhead) load(i);
    float xhat[C][V], h[C][V], s = 0.0f, q = 0.0f;
    const float r = rstd;
    const bool there = i < a.m;
    float w[C][V];  // from L1 or L2 for each row: kept, they would not leave registers for the next row's loads
    load_vector<V>(a.weight, k, 1.0f, w);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float ge = (float)g.e[c][e];
        xhat[c][e] = ((float)x.e[c][e] - mean) * rstd;
        h[c][e] = ge * w[c][e];
        s += e >= k.skip[c] ? h[c][e] : 0.0f;
        q += e >= k.skip[c] ? h[c][e] * xhat[c][e] : 0.0f;
        if (there) {
          dw[c][e] = fmaf(ge, xhat[c][e], dw[c][e]);
          db[c][e] += ge;
        }
      }
    if (kAhead && i0 + step < a.m) load(i + step);
    s = group_sum(s, kGroup);
    q = group_sum(q, kGroup);
    if constexpr (kWaves > 1) {
      if (lane == 0) {
        part[turn][0][threadIdx.x / 64] = s;
        part[turn][1][threadIdx.x / 64] = q;
      }
      __syncthreads();
      s = row_sum<kWaves>(part[turn][0], sub * kWaves);
      q = row_sum<kWaves>(part[turn][1], sub * kWaves);
    }
    if (!there || !a.dx) continue;
    s *= inv_n;
    q *= inv_n;
    T* dx = static_cast<T*>(a.dx) + i * a.lddx;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (k.skip[c] == V) continue;
      T o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = (T)(r * (h[c][e] - s - xhat[c][e] * q));
      __builtin_memcpy(dx + k.at[c], o, 16);
    }
  }
  if (!a.sums) return;
  // columns of chunk c: L V neighbours from c L V on, V of each of the first row's threads
  float* sums = a.sums + (int64_t)blockIdx.x * 2 * a.n;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) join[sub][t * V + e] = which ? db[c][e] : dw[c][e];
      __syncthreads();
      for (int col = threadIdx.x; col < L * V; col += kGradientThreads) {
        const int64_t j = (int64_t)c * L * V + col;
        if (j >= a.n) break;
        // the last, shifted chunk: column j lies skip elements further into it
        const int64_t last = a.n - V, first = j / V * V;
        const int from = first > last ? col + (int)(first - last) : col;
        float s = join[0][from];
#pragma unroll
        for (int r = 1; r < kRows; ++r) s += join[r][from];
        sums[which * a.n + j] = s;
      }
    }
}

// The sum of either type over a workgroup.
template <int kThreads>
using RowSum = std::conditional_t<kThreads == 64, float, double>;
template <int kThreads>
__device__ __forceinline__ RowSum<kThreads> block_sum(RowSum<kThreads> x, RowSum<kThreads>* lds) {
  if constexpr (kThreads == 64) return group_sum(x, 64);
  else return wide_sum<kThreads>(x, lds);
}

// Rows of any length: the sums and dX of a row by one workgroup, which walks it twice. The sums of long ones are fp64, four terms
// at a time in fp32. (us, 2000 x 32768 of bf16: 265, each term in fp64 345, all in fp32 251.)
template <typename T, int kThreads>
__global__ __launch_bounds__(kThreads) void norm_gradient_any(NormGradientArgs a) {
  typedef RowSum<kThreads> Sum;
  __shared__ Sum lds[kThreads / 64];
  for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    const T* g = static_cast<const T*>(a.g) + i * a.ldg;
    T* dx = static_cast<T*>(a.dx) + i * a.lddx;
    const float mean = a.mean[i], rstd = a.rstd[i];
    Sum all_h = 0, all_hx = 0;
    constexpr int kBatch = kThreads == 64 ? 1 : 4;
    for (int64_t j0 = threadIdx.x; j0 < a.n; j0 += kBatch * kThreads) {
      float some_h = 0.0f, some_hx = 0.0f;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const bool there = j0 + u * kThreads < a.n;
        const int64_t j = there ? j0 + u * kThreads : j0;
        const float h = (float)g[j] * (a.weight ? a.weight[j] : 1.0f), hx = h * (((float)x[j] - mean) * rstd);
        some_h += there ? h : 0.0f;
        some_hx += there ? hx : 0.0f;
      }
      all_h += (Sum)some_h;
      all_hx += (Sum)some_hx;
    }
    const float s = (float)(block_sum<kThreads>(all_h, lds) / (Sum)a.n), q = (float)(block_sum<kThreads>(all_hx, lds) / (Sum)a.n);
    for (int64_t j = threadIdx.x; j < a.n; j += kThreads) {
      const float h = (float)g[j] * (a.weight ? a.weight[j] : 1.0f);
      dx[j] = (T)(rstd * (h - s - ((float)x[j] - mean) * rstd * q));
    }
  }
}

// Their column sums: a thread owns a column over every groups-th row.
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_any(NormGradientArgs a) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= a.n) return;
  const T* X = static_cast<const T*>(a.x) + j;
  const T* G = static_cast<const T*>(a.g) + j;
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t i = blockIdx.y; i < a.m; i += a.groups) {
    const float g = (float)G[i * a.ldg];
    dw = fmaf(g, ((float)X[i * a.ldx] - a.mean[i]) * a.rstd[i], dw);
    db += g;
  }
  a.sums[(int64_t)blockIdx.y * 2 * a.n + j] = dw;
  a.sums[((int64_t)blockIdx.y * 2 + 1) * a.n + j] = db;
}

// dweight and dbias from the workgroups' sums [groups][2][n], in fp64 and in a fixed order: 16 columns of the
// 2 n a workgroup at a time, as in column_sum.
__global__ __launch_bounds__(256) void norm_gradient_finish(NormGradientArgs a) {
  __shared__ double lds[256];
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  for (int64_t j0 = (int64_t)blockIdx.x * 16; j0 < 2 * a.n; j0 += (int64_t)gridDim.x * 16) {
    const int64_t j = j0 + c;
    double s = 0.0;
    if (j < 2 * a.n) {
#pragma unroll 4
      for (int64_t g = slot; g < a.groups; g += 16) s += (double)a.sums[g * 2 * a.n + j];
    }
    lds[threadIdx.x] = s;
    __syncthreads();
    if (slot == 0 && j < 2 * a.n) {
      for (int p = 1; p < 16; ++p) s += lds[p * 16 + c];
      float* out = j < a.n ? a.dweight : a.dbias;
      if (out) out[j < a.n ? j : j - a.n] = (float)s;
    }
    __syncthreads();
  }
}

constexpr int64_t kMostGroups = 256;  // one workgroup per CU

template <typename T, int L, bool kStreamed>
void norm_launch(const NormArgs& a, unsigned grid, hipStream_t s) {
  constexpr int kBlock = L < 256 ? 256 : L;
  const int64_t chunks = (a.n + kChunkOf<T> - 1) / kChunkOf<T>;
  if constexpr (L == 16) {  // more threads come with more chunks than threads
    if (chunks <= L) return norm_rows<T, L, 1, kStreamed><<<grid, kBlock, 0, s>>>(a);
  }
  if (chunks <= 2 * L) norm_rows<T, L, 2, kStreamed><<<grid, kBlock, 0, s>>>(a);
  else norm_rows<T, L, 4, kStreamed><<<grid, kBlock, 0, s>>>(a);
}

// Workgroups: enough rows under way, few enough that they keep weight and bias. us, with 2, 4 and 8 (of 1024 threads 1, 2, 4)
// a CU: 16384 x 4096 of bf16 50, 53, 54, streamed 49, 51, 52; 4000 x 16384 51, 53, 58, streamed 49 with 2; one
// workgroup a row 56, 71. Rows of a wavefront or less: 9.5, 9.2, 9.1 at 40000 x 256.
template <typename T, int L>
void norm_for(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = L < 256 ? 256 / L : 1;
  const int64_t most = L < 256 ? 1024 : 512, groups = (a.m + kRows - 1) / kRows;
  const unsigned grid = (unsigned)(groups < most ? groups : most);
  if (a.m * a.n * (int64_t)sizeof(T) > kL2Bytes) norm_launch<T, L, true>(a, grid, s);
  else norm_launch<T, L, false>(a, grid, s);
}

// Threads of a row: the fewest of 16, 64, 256 and 1024 with up to four chunks each. us with these, and with twice or half as
// many: bf16 40000 x 256 9.4, 10.5; 30000 x 500 12.6, 11.1; 20000 x 768 12.9, 13.5 with half, 17.8; 10392 x 1269 13.6, 14.5;
// 16384 x 2048 24.2, 22.5; 16384 x 4096 47.6, 53.1 with half, 58.1; 8192 x 5120 34.1, 33.5; 4000 x 12000 42.9, 37.5 with half;
// 4000 x 16384 49.0, 49.2 with half; fp32 40000 x 250 17.1, 14.6; 8192 x 768 9.9, 10.3; 5001 x 1111 12.8, 10.0 with half; 4000 x
// 4000 20.9, 21.0; 4000 x 6000 38.6, 33.2 with half. So every power of two would serve some widths better; with these four
// a call takes up to 29% longer than with the best.
template <typename T>
void norm_type(const NormArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  if (a.n < V || a.n > 1024 * 4 * V) {
    const unsigned grid = (unsigned)(a.m < 4096 ? a.m : 4096);
    if (a.n < V) norm_short<T><<<grid, 64, 0, s>>>(a);
    else norm_long<T><<<grid, 1024, 0, s>>>(a);
  } else if (a.n <= 16 * 4 * V) {
    norm_for<T, 16>(a, s);
  } else if (a.n <= 64 * 4 * V) {
    norm_for<T, 64>(a, s);
  } else if (a.n <= 256 * 4 * V) {
    norm_for<T, 256>(a, s);
  } else {
    norm_for<T, 1024>(a, s);
  }
}

template <typename T, int L>
void norm_gradient_for(const NormGradientArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  const int64_t chunks = (a.n + V - 1) / V;
  const unsigned grid = (unsigned)a.groups;
  if constexpr (L == 16) {
    if (chunks <= L) return norm_gradient_rows<T, L, 1><<<grid, kGradientThreads, 0, s>>>(a);
  }
  if constexpr (L == 1024 && V == 4) {
    if (chunks > 2 * L) return norm_gradient_rows<T, L, 4><<<grid, kGradientThreads, 0, s>>>(a);
  }
  norm_gradient_rows<T, L, 2><<<grid, kGradientThreads, 0, s>>>(a);
}

// Threads of a row, the fewest with up to two chunks each (fp32 rows of more than 8192: four): a second chunk keeps more loads
// under way. us with twice the threads and one chunk: bf16 16384 x 2048 50, two 46; 16384 x 5120 144, 116; fp32 20000 x 768
// 44, 40; 8000 x 2560 68, 51.
int norm_gradient_lanes(int64_t n, int chunk) {
  int lanes = 16;
  while (lanes < 1024 && n > 2 * lanes * chunk) lanes *= 2;
  return lanes;
}

template <typename T>
void norm_gradient_type(const NormGradientArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  if (a.n < V || a.n > kNormGradientMost) {
    const unsigned grid = (unsigned)(a.m < 4096 ? a.m : 4096);
    if (a.dx && a.n < V) norm_gradient_any<T, 64><<<grid, 64, 0, s>>>(a);
    else if (a.dx) norm_gradient_any<T, 1024><<<grid, 1024, 0, s>>>(a);
    if (a.sums) norm_columns_any<T><<<dim3((unsigned)((a.n + 255) / 256), (unsigned)a.groups), 256, 0, s>>>(a);
  } else {
    switch (norm_gradient_lanes(a.n, V)) {
      case 16: norm_gradient_for<T, 16>(a, s); break;
      case 32: norm_gradient_for<T, 32>(a, s); break;
      case 64: norm_gradient_for<T, 64>(a, s); break;
      case 128: norm_gradient_for<T, 128>(a, s); break;
      case 256: norm_gradient_for<T, 256>(a, s); break;
      case 512: norm_gradient_for<T, 512>(a, s); break;
      default: norm_gradient_for<T, 1024>(a, s); break;
    }
  }
  const int64_t finish = (2 * a.n + 15) / 16, most = 1 << 20;  // threads of a launch stay below 2^32
  if (a.sums) norm_gradient_finish<<<(unsigned)(finish < most ? finish : most), 256, 0, s>>>(a);
}

}  // namespace

int64_t norm_gradient_groups(int64_t m, int64_t n, int type) {
  // rows that a workgroup takes at once; the kernels for any length take one
  const int chunk = 16 / elem_size(type);
  const int64_t rows = n > kNormGradientMost || n < chunk ? 1 : kGradientThreads / norm_gradient_lanes(n, chunk);
  const int64_t groups = (m + rows - 1) / rows;
  return groups < kMostGroups ? groups : kMostGroups;
}

hipError_t launch_norm(const NormArgs& a, int type, hipStream_t s) {
  if (type == kBf16) norm_type<__bf16>(a, s);
  else if (type == kF16) norm_type<_Float16>(a, s);
  else norm_type<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_norm_gradient(const NormGradientArgs& a, int type, hipStream_t s) {
  if (type == kBf16) norm_gradient_type<__bf16>(a, s);
  else if (type == kF16) norm_gradient_type<_Float16>(a, s);
  else norm_gradient_type<float>(a, s);
  return hipGetLastError();
}

}  // namespace xtvxy
