// Softmax cross entropy and distillation over the classes of an output layer, without keeping its logits.
//
//     t_ij = (sum_k x_ik w_jk + bias_j) / T,  lse_i = log sum_j exp(t_ij),
//     labels y:             loss_i = lse_i - t_i,y                                    target_ij = [j = y_i]
//     a teacher's weights P: loss_i = sum_c P_ic (log P_ic - t_ic + lse_i)            target_ij = P_ij
//     d_ij = grad_i / T (exp(t_ij - lse_i) - target_ij),  dX = d W,  dW = d^T X,  dbias_j = sum_i d_ij.
//
// The products run through the ring kernel (linear_ring.h) and are what bounds both directions; what happens to the
// logits happens in a tile's registers. Forward: each wavefront reduces its half of a tile's columns to the largest t
// and the sum of exp(t - largest) per row, and writes down t of the classes that its rows list; the sums of all tiles
// are joined in a fixed order. Gradient: the logits are formed once more, piece by piece of the vocabulary (a
// fourth product; keeping them costs as much memory as the vocabulary is wide), turned into d, and the piece's d,
// in the element type, goes through the layer's gradient kernel.
//
// Tiles are the product's: of 256 x 256 the product over 1000 features takes 26 us, first loads and epilogue 15 to 20, in
// which the matrix unit waits. us: bf16 8192 x 2048 x 65536 forward 1590 to 1660 from card to card (1.39 to 1.33 PFLOP/s, matrix
// unit 68% busy), with the gradient 6600; fp16 2047 x 1000 x 30001 with 32 classes a row 610 with the gradient (186 forward,
// 182 d, 232 its products); fp32 512 x 768 x 16384 100 (fp32 matrix unit 89% busy). Few rows are bound by W: fp16 13 x 4096 x
// 32000 60, of which its one pass 51 (5.2 TB/s).
#include "linear_ring.h"
#include "loss.h"

namespace xtvxy {
namespace {

__device__ __forceinline__ int64_t class_at(const ClassList& l, int64_t i, int e) {
  const int64_t at = i * l.ld + e;
  return l.bits == 32 ? static_cast<const int32_t*>(l.p)[at] : static_cast<const int64_t*>(l.p)[at];
}

// For every class that a strip's rows list within its columns: fn(row of the strip, its place in the list, place of its
// value in the staging area). Short lists are searched, lanes taking their entries in turn; of long ones the tile has the
// entries by strip and half tile: searching 32 a row took 30 us a 256 x 256 tile, as long as its product at k = 1000.
template <int WN, typename Fn>
__device__ __forceinline__ void for_listed(const ClassList& list, const ListOrder& order, int64_t i0, int rows,
                                           int64_t first_class, int columns, Fn fn) {
  const uint32_t per_row = (uint32_t)list.per_row, lane = threadIdx.x & 63;
  if (columns <= 0) return;
  if (order.starts) {
    const int64_t strip = i0 / order.strip_rows;
    const uint32_t* starts = order.starts + strip * (order.columns + 1) + first_class / WN;
    const uint32_t* entries = order.entries + strip * order.strip_rows * per_row;
    const uint32_t end = starts[1];
    for (uint32_t at = starts[0] + lane; at < end; at += 64) {
      const uint32_t e = entries[at];
      const int row = (int)(e & 63), c = (int)(e >> 6 & 127);
      fn(row, (int)(e >> 13), staged_at<WN>(row, c >> 2) + (c & 3));
    }
    return;
  }
  constexpr int kBatch = 4;
  const uint32_t total = (uint32_t)rows * per_row;
  for (uint32_t at0 = lane; at0 < total; at0 += 64 * kBatch) {
    int64_t c[kBatch];
    uint32_t row[kBatch], e[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const uint32_t at = at0 + b * 64 < total ? at0 + b * 64 : at0;
      row[b] = per_row == 1 ? at : at / per_row;
      e[b] = at - row[b] * per_row;
      c[b] = class_at(list, i0 + row[b], (int)e[b]) - first_class;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (at0 + b * 64 < total && c[b] >= 0 && c[b] < columns)
        fn((int)row[b], (int)e[b], staged_at<WN>((int)row[b], (int)c[b] >> 2) + ((int)c[b] & 3));
  }
}

// Whether there may be any: labels and ordered lists are looked at, other lists are short.
template <int WN>
__device__ __forceinline__ bool any_listed(const ClassList& list, const ListOrder& order, int64_t i0, int rows, int64_t first_class,
                                           int columns) {
  if (columns <= 0) return false;
  if (order.starts) {
    const uint32_t* starts = order.starts + i0 / order.strip_rows * (order.columns + 1) + first_class / WN;
    return starts[0] != starts[1];
  }
  if (list.per_row > 1) return true;
  const int lane = threadIdx.x & 63;
  const int64_t c = lane < rows ? class_at(list, i0 + lane, 0) - first_class : -1;
  return __any(c >= 0 && c < columns);
}

// A workgroup puts a strip's entries in order: counted by half tile, the counts summed, and placed. Entries of one half tile
// come in any order: each has a value of its own.
constexpr int kOrderThreads = 1024;
__global__ __launch_bounds__(kOrderThreads) void list_order(OrderArgs a) {
  __shared__ uint32_t count[kMostHalves];
  __shared__ uint32_t totals[kOrderThreads / 64];
  const int64_t strip = blockIdx.x, i0 = strip * a.order.strip_rows;
  const int columns = (int)a.order.columns, per_row = a.list.per_row;
  const int rows = a.m - i0 < a.order.strip_rows ? (int)(a.m - i0) : a.order.strip_rows;
  uint32_t* starts = a.order.starts + strip * (columns + 1);
  uint32_t* entries = a.order.entries + strip * a.order.strip_rows * per_row;
  for (int h = threadIdx.x; h < columns; h += kOrderThreads) count[h] = 0;
  __syncthreads();
  const int half_bits = 31 - __builtin_clz(a.order.half);
  const auto each = [&](auto fn) {
    constexpr int kBatch = 4;
    for (int at0 = threadIdx.x; at0 < rows * per_row; at0 += kBatch * kOrderThreads) {
      int64_t c[kBatch];
      int row[kBatch], e[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int at = at0 + b * kOrderThreads < rows * per_row ? at0 + b * kOrderThreads : at0;
        row[b] = at / per_row;
        e[b] = at - row[b] * per_row;
        c[b] = class_at(a.list, i0 + row[b], e[b]);
        if (a.weights && a.weights[(i0 + row[b]) * per_row + e[b]] == 0.0f) c[b] = -1;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (at0 + b * kOrderThreads < rows * per_row && c[b] >= 0 && c[b] < a.n)
          fn(row[b], e[b], (int)(c[b] >> half_bits), (int)c[b] & (a.order.half - 1));
    }
  };
  each([&](int, int, int half, int) { atomicAdd(&count[half], 1u); });
  __syncthreads();
  // each thread sums neighbours, the threads' sums join over the wavefronts
  const int share = (columns + kOrderThreads - 1) / kOrderThreads, h0 = threadIdx.x * share, lane = threadIdx.x & 63;
  uint32_t own = 0;
  for (int h = h0; h < h0 + share && h < columns; ++h) own += count[h];
  uint32_t sum = own;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) {
    const uint32_t v = __shfl_up(sum, by);
    if (lane >= by) sum += v;
  }
  if (lane == 63) totals[threadIdx.x >> 6] = sum;
  __syncthreads();
  uint32_t before = sum - own;
  for (int w = 0; w < kOrderThreads / 64; ++w)
    if (w < (int)(threadIdx.x >> 6)) before += totals[w];
  for (int h = h0; h < h0 + share && h < columns; ++h) {
    const uint32_t c = count[h];
    starts[h] = count[h] = before;
    before += c;
  }
  if (threadIdx.x == kOrderThreads - 1) starts[columns] = before;
  __syncthreads();
  each([&](int row, int e, int half, int column) {
    entries[atomicAdd(&count[half], 1u)] = (uint32_t)row | (uint32_t)column << 6 | (uint32_t)e << 13;
  });
}

// The bias over T of a lane's columns, four neighbours of each of the FB groups of 16; -infinity where there is no
// column, whose product is zero.
template <int FB>
__device__ __forceinline__ void lane_bias(const float* bias, float inv_temperature, int64_t j, int64_t n, f32x4 (&b)[FB]) {
#pragma unroll
  for (int y = 0; y < FB; ++y) {
    const int64_t at = j + y * 16;
    b[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (bias && at < n) b[y] = load4<float>(bias + at, n - at >= 4 ? 4 : (int)(n - at)) * inv_temperature;
    if (at + 4 > n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[y][e] = at + e < n ? b[y][e] : -__builtin_inff();
    }
  }
}

// t = z / T + bias / T of one row's columns of a lane.
template <int FB>
__device__ __forceinline__ void lane_logits(const f32x4 (&z)[FB], const f32x4 (&bias)[FB], float inv_temperature, f32x4 (&t)[FB]) {
#pragma unroll
  for (int y = 0; y < FB; ++y)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[y][e] = fmaf(z[y][e], inv_temperature, bias[y][e]);
}

// Of 16-bit features without a bias, in whole tiles, exp(t - u) is exp2(z c - ref), c = log2 e / T and ref = u log2 e: one
// operation less than the difference with the bias and its product with log2 e. What the roundings of c and ref leave, 2^-23
// |u|, is nearly alike in all of a row's logits that count, those next to u: one factor a row takes it out. Beyond
// kFarLogit ref's rounding would leave no distance (at 1e11 it was thousands). The factors cost nothing that shows (us with
// and without, with the gradient: bf16 8192 x 2048 x 65536 6656, 6661; 2048 x 256 x 32768 242.9, 242.0). fp32 takes the exact
// difference, at 0.1 to 0.5% (1024 x 512 x 32768 with the gradient 773.7, 772.9).
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f, kFarLogit = 1e6f;
struct Log2Scale {
  float c, rest;  // rest: what c's rounding takes off the product with T u, per u
  __device__ __forceinline__ explicit Log2Scale(float inv_temperature)
      : c(inv_temperature * kLog2e), rest(fmaf(inv_temperature, kLog2e, -c) / inv_temperature) {}
  // of exp2(z c - ref), z next to T u: the constant log2 e's own rounding is in both and cancels
  __device__ __forceinline__ float correction(float u, float ref) const {
    return __builtin_amdgcn_exp2f(fmaf(u, rest, -fmaf(u, kLog2e, -ref)));
  }
};

__device__ __forceinline__ float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

struct StatsEnd {
  const LossForwardArgs& l;
  template <typename T, int BM, int BN, typename S>
  __device__ __forceinline__ void finish(const ProductArgs& a, uint8_t* ring, S& sums, const TilePlace& p) const {
    constexpr int FA = BM / 32, FB = BN / 32;
    typedef Strips<BM, BN> Strip;
    constexpr int WN = Strip::kWidth, kRows = Strip::kRows;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wi = (wave >> 1) * (BM / 2), wj = (wave & 1) * (BN / 2), r = lane & 15, g = lane >> 4;
    f32x4 bias[FB];
    lane_bias<FB>(l.bias, l.inv_temperature, p.j0 + wj + g * 4, a.n, bias);
    end_of_products(sums);
    float* stats = l.stats + (p.j0 / BN * 2 + (wave & 1)) * a.m * 2;
    const bool plain = sizeof(T) == 2 && !l.bias && p.j0 + BN <= a.n;
    const Log2Scale log2(l.inv_temperature);
#pragma unroll
    for (int x = 0; x < FA; ++x) {
      const f32x4(&z)[FB] = sums.acc[x];
      float top = 0.0f, s = 0.0f;
      bool done = false;
      if (plain) {
        top = z[0][0];
#pragma unroll
        for (int y = 0; y < FB; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, z[y][e]);
        const float ref = max_xor32(max_xor16(top)) * log2.c;
        done = __all(fabsf(ref) < kFarLogit);
        if (done) {
#pragma unroll
          for (int y = 0; y < FB; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(fmaf(z[y][e], log2.c, -ref));
          top = ref * kLn2;
          s *= log2.correction(top, ref);
        }
      }
      if (!done) {
        f32x4 t[FB];
        lane_logits<FB>(z, bias, l.inv_temperature, t);
        top = t[0][0];
#pragma unroll
        for (int y = 0; y < FB; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, t[y][e]);
        top = max_xor32(max_xor16(top));
        // a row without a finite logit here has no distances from its largest one
        const float from = top == -__builtin_inff() ? 0.0f : top;
        s = 0.0f;
#pragma unroll
        for (int y = 0; y < FB; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s += fast_exp(t[y][e] - from);
      }
      s = add_xor32(add_xor16(s));
      const int64_t i = p.i0 + wi + x * 16 + r;
      if (g == 0 && i < a.m) *reinterpret_cast<f32x2*>(stats + i * 2) = f32x2{top, s};
    }
    if (l.list.per_row == 0) return;
    float* area = reinterpret_cast<float*>(ring + wave * Strip::kArea);
    const int64_t width = a.n - p.j0 - wj;
#pragma unroll
    for (int part = 0; part < BM / 2 / kRows; ++part) {
      const int64_t i0 = p.i0 + wi + part * kRows;
      if (i0 >= a.m) break;
      const int rows = a.m - i0 < kRows ? (int)(a.m - i0) : kRows, columns = width < WN ? (int)width : WN;
      // most strips of a wide vocabulary hold none of their rows' classes
      if (!any_listed<WN>(l.list, l.order, i0, rows, l.first_class + p.j0 + wj, columns)) continue;
#pragma unroll
      for (int x = part * kRows / 16; x < (part + 1) * kRows / 16; ++x) {
        f32x4 t[FB];
        lane_logits<FB>(sums.acc[x], bias, l.inv_temperature, t);
#pragma unroll
        for (int y = 0; y < FB; ++y) *reinterpret_cast<f32x4*>(area + staged_at<WN>(x * 16 % kRows + r, y * 4 + g)) = t[y];
      }
      __builtin_amdgcn_wave_barrier();
      for_listed<WN>(l.list, l.order, i0, rows, l.first_class + p.j0 + wj, columns,
                     [&](int row, int e, int at) { l.listed[(i0 + row) * l.list.per_row + e] = area[at]; });
      __builtin_amdgcn_wave_barrier();
    }
  }
};

// d is stored in the type of the features: the matrix instructions of its two products take both operands in one type, and the
// layer's gradient rounds its own d alike. What that costs 16-bit dX and dW, in the 2-norm: bf16 1.64e-3 (their own
// rounding) to 2.22e-3, fp16 2.1e-4 to 2.9e-4, where rows have unlike factors (alike: see LossFactorArgs). A d of two
// 16-bit parts would double the work of the products, which are half of the time. Column sums take it in fp32.
struct GradientEnd {
  const LossGradientArgs& l;
  template <typename T, int BM, int BN, typename S>
  __device__ __forceinline__ void finish(const ProductArgs& a, uint8_t* ring, S& sums, const TilePlace& p) const {
    constexpr int FA = BM / 32, FB = BN / 32;
    typedef Strips<BM, BN> Strip;
    constexpr int WN = Strip::kWidth, kRows = Strip::kRows, kLanes = WN / 8, kStep = 64 / kLanes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wi = (wave >> 1) * (BM / 2), wj = (wave & 1) * (BN / 2), r = lane & 15, g = lane >> 4;
    f32x4 bias[FB];
    lane_bias<FB>(l.bias, l.inv_temperature, p.j0 + wj + g * 4, a.n, bias);
    float factors[FA], norms[FA];
    bool near = true;
#pragma unroll
    for (int x = 0; x < FA; ++x) {
      const int64_t i = p.i0 + wi + x * 16 + r;
      factors[x] = i < a.m ? l.factor[i] : 0.0f;
      norms[x] = i < a.m ? l.lse[i] : 0.0f;
      near &= fabsf(norms[x]) < kFarLogit;
    }
    end_of_products(sums);
    const Log2Scale log2(l.inv_temperature);
    const bool plain = sizeof(T) == 2 && !l.bias && p.j0 + BN <= a.n && log2.c < __builtin_inff() && __all(near);
    float* area = reinterpret_cast<float*>(ring + wave * Strip::kArea);
    const int64_t width = a.n - p.j0 - wj;
    const int c8 = lane % kLanes;
    const int64_t column = p.j0 + wj + c8 * 8;  // of this lane's eight
    constexpr bool kScaled = sizeof(T) == 2;
    const float scale = kScaled && l.scale ? *l.scale : 1.0f;
    float column_sums[8] = {};
#pragma unroll
    for (int part = 0; part < BM / 2 / kRows; ++part) {
      const int64_t i0 = p.i0 + wi + part * kRows;
      if (i0 >= a.m) break;
      const int rows = a.m - i0 < kRows ? (int)(a.m - i0) : kRows;
#pragma unroll
      for (int x = part * kRows / 16; x < (part + 1) * kRows / 16; ++x) {
        const float factor = factors[x];
        f32x4 d[FB];
        if (plain) {
          const float ref = norms[x] * kLog2e;
          const float near_factor = factor * log2.correction(norms[x], ref);
#pragma unroll
          for (int y = 0; y < FB; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[y][e] = near_factor * __builtin_amdgcn_exp2f(fmaf(sums.acc[x][y][e], log2.c, -ref));
        } else {
          lane_logits<FB>(sums.acc[x], bias, l.inv_temperature, d);
#pragma unroll
          for (int y = 0; y < FB; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[y][e] = factor * fast_exp(d[y][e] - norms[x]);
        }
#pragma unroll
        for (int y = 0; y < FB; ++y) {
#pragma unroll
          for (int e = 0; e < 4; ++e)  // a row that does not count is zero whatever its logits are
            d[y][e] = factor == 0.0f ? 0.0f : d[y][e];
          *reinterpret_cast<f32x4*>(area + staged_at<WN>(x * 16 % kRows + r, y * 4 + g)) = d[y];
        }
      }
      __builtin_amdgcn_wave_barrier();
      for_listed<WN>(l.list, l.order, i0, rows, l.first_class + p.j0 + wj, width < WN ? (int)width : WN, [&](int row, int e, int at) {
        const float factor = l.factor[i0 + row], w = l.weights ? l.weights[(i0 + row) * l.list.per_row + e] : 1.0f;
        // a class that is listed twice comes here twice, maybe at once
        if (factor != 0.0f && w != 0.0f) __hip_atomic_fetch_add(area + at, -factor * w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      });
      __builtin_amdgcn_wave_barrier();
      if (column < l.ldd) {
        T* d = static_cast<T*>(l.d) + (l.d ? i0 * l.ldd + column : 0);
#pragma unroll 4
        for (int row = lane / kLanes; row < rows; row += kStep) {
          const f32x8 v = staged8<WN>(area, row, c8);
          typename Vec<T>::x8 o;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            column_sums[e] += v[e];
            o[e] = (T)(kScaled ? v[e] * scale : v[e]);
          }
          if (l.d) *reinterpret_cast<typename Vec<T>::x8*>(d + row * l.ldd) = o;
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    if (!l.sums) return;
    float* out = l.sums + (p.i0 / BM * 2 + (wave >> 1)) * a.n;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int by = kLanes; by < 64; by *= 2) column_sums[e] += __shfl_xor(column_sums[e], by);
    }
    const int count = a.n - column >= 8 ? 8 : (a.n > column ? (int)(a.n - column) : 0);
    if (lane < kLanes && count > 0) store_elems<float, 8>(out + column, count, column_sums);
  }
};

template <typename T, int TILE, typename End>
__device__ __forceinline__ void loss_tile(const ProductArgs& a, uint8_t* ring, const End& end) {
  if constexpr (TILE == 256) ring_tile_halves<T, TILE, TILE, false, false>(a, blockIdx.x, ring, end);
  else ring_tile<T, TILE, TILE, false, false>(a, blockIdx.x, ring, end);
}

template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void loss_forward(LossForwardArgs a) {
  __shared__ __align__(1024) uint8_t ring[ring_bytes(TILE)];
  loss_tile<T, TILE>(a.product, ring, StatsEnd{a});
}

// t of up to four neighbouring classes of a row of logits in memory (the parts of a split product, which it adds).
__device__ __forceinline__ f32x4 few_logits(const LossForwardArgs& a, int64_t i, int64_t j, int count) {
  const ProductArgs& p = a.product;
  const float none = -__builtin_inff();
  if (count <= 0) return f32x4{none, none, none, none};
  const float* z = p.partial + i * p.n + j;
  f32x4 t = load4<float>(z, count);
  for (int q = 1; q < p.splits; ++q) t += load4<float>(z + q * p.m * p.n, count);
  const f32x4 b = a.bias ? load4<float>(a.bias + j, count) * a.inv_temperature : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = e < count ? fmaf(t[e], a.inv_temperature, b[e]) : none;
  return t;
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int by = 1; by < 16; by *= 2) x = fmaxf(x, __shfl_xor(x, by));
  return max_xor32(max_xor16(x));
}

// A workgroup takes 4096 classes of a row; its largest t and sum through LDS.
__global__ __launch_bounds__(256) void loss_few(LossForwardArgs a) {
  __shared__ float tops[4], sums[4];
  constexpr int kQuads = kFewChunk / 4 / 256;
  const ProductArgs& p = a.product;
  const int64_t i = blockIdx.y, j0 = (int64_t)blockIdx.x * kFewChunk;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  f32x4 t[kQuads];
  float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    const int64_t j = j0 + (q * 256 + threadIdx.x) * 4;
    t[q] = few_logits(a, i, j, p.n - j >= 4 ? 4 : (int)(p.n > j ? p.n - j : 0));
  }
#pragma unroll
  for (int q = 0; q < kQuads; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, t[q][e]);
  top = wave_max(top);
  if (lane == 0) tops[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, tops[w]);
  const float from = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
  for (int q = 0; q < kQuads; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += fast_exp(t[q][e] - from);
  sum = group_sum(sum, 64);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) *reinterpret_cast<f32x2*>(a.stats + ((int64_t)blockIdx.x * p.m + i) * 2) = f32x2{top, sums[0] + sums[1] + sums[2] + sums[3]};
  for (int e = threadIdx.x; e < a.list.per_row; e += 256) {
    const int64_t c = class_at(a.list, i, e) - a.first_class;
    if (c >= j0 && c < j0 + kFewChunk && c < p.n) a.listed[i * a.list.per_row + e] = few_logits(a, i, c, 1)[0];
  }
}

template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void loss_gradient(LossGradientArgs a) {
  __shared__ __align__(1024) uint8_t ring[ring_bytes(TILE)];
  loss_tile<T, TILE>(a.product, ring, GradientEnd{a});
}

// (largest, sum of exp(t - largest)) of two sets of logits joined. Either may be empty: (-infinity, 0).
__device__ __forceinline__ void join_stats(float* top, float* sum, float top2, float sum2) {
  const float t = fmaxf(*top, top2), from = t == -__builtin_inff() ? 0.0f : t;
  *sum = *sum * fast_exp(*top - from) + sum2 * fast_exp(top2 - from);
  *top = t;
}

__device__ __forceinline__ float teacher_at(const TeacherArgs& a, int64_t at) {
  if (a.type == kBf16) return (float)static_cast<const __bf16*>(a.teacher)[at];
  if (a.type == kF16) return (float)static_cast<const _Float16*>(a.teacher)[at];
  return static_cast<const float*>(a.teacher)[at];
}

// A row's weight as stored: a class beyond the vocabulary or an infinite or missing logit makes the whole row no distribution.
__device__ __forceinline__ float stored_weight(bool bad, float sum, float w) {
  return bad || !(sum < __builtin_inff()) ? __builtin_nanf("") : w;
}

// Whether two of a wavefront's valid classes are equal. Lanes write themselves into the place of their class; who finds
// another class there tries again without those that found themselves. `places`: 256 bytes of LDS of the wavefront.
__device__ __forceinline__ bool any_equal(int32_t c, bool valid, volatile uint8_t* places) {
  const int lane = threadIdx.x & 63, place = (int)((uint32_t)c * 2654435761u >> 24);
  bool open = valid, equal = false;
  while (__any(open)) {
    if (open) places[place] = (uint8_t)lane;
    __builtin_amdgcn_wave_barrier();
    const int who = open ? places[place] : lane;
    __builtin_amdgcn_wave_barrier();
    equal |= __shfl(c, who) == c && who != lane;
    open = open && who != lane && !equal;
  }
  return __any(equal);
}

// The weights of a row of up to kLaneListed classes, by a wavefront. (Comparing every two places takes 0.2 us a place of
// 4575 rows.)
__device__ __forceinline__ void teacher_row(const TeacherArgs& a, int64_t i, volatile uint8_t* places) {
  const int lane = threadIdx.x & 63, count = a.list.per_row;
  const int64_t at = lane < count ? class_at(a.list, i, lane) : -1;
  const bool valid = at >= 0 && at < a.n;
  const int32_t c = valid ? (int32_t)at : -1;
  const float t = valid ? teacher_at(a, i * a.ldt + lane) * a.inv_temperature : -__builtin_inff();
  const bool bad = __any(at >= a.n || t != t);
  float top = t;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) top = fmaxf(top, __shfl_xor(top, by));
  const float own = expf(t - (top == -__builtin_inff() ? 0.0f : top)), sum = group_sum(own, 64);
  float w = own;
  bool first = true;
  if (any_equal(c, valid, places)) {
    w = 0.0f;
    for (int f = 0; f < count; ++f) {
      const bool same = __builtin_amdgcn_readlane(c, f) == c;
      if (same && f < lane) first = false;
      if (same && f >= lane) w += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, own), f));
    }
  }
  if (lane < count) a.weights[i * count + lane] = stored_weight(bad, sum, first && valid && sum > 0.0f ? w / sum : 0.0f);
}

// 16 rows a workgroup: of each row a thread joins every 64th part's statistics, the 64 join in order; the terms of a
// teacher's classes likewise. (With 16 threads a row 1000 parts of 13 rows took 9.6 us.)
constexpr int kSlots = 64;
__global__ __launch_bounds__(16 * kSlots) void loss_finish(LossFinishArgs a) {
  __shared__ float tops[kSlots][17], sums[kSlots][17], terms[kSlots][17], norms[16];
  __shared__ uint8_t places[16][256];
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int64_t i = (int64_t)blockIdx.x * 16 + c;
  const bool there = i < a.m;
  if (a.last && a.teacher.teacher) {  // a wavefront a row
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 6);
    if (row < a.m) teacher_row(a.teacher, row, places[threadIdx.x >> 6]);
  }
  float top = -__builtin_inff(), sum = 0.0f;
  if (there) {
    for (int64_t p = slot; p < a.parts; p += 4 * kSlots) {
      f32x2 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool part = p + u * kSlots < a.parts;
        v[u] = *reinterpret_cast<const f32x2*>(a.stats + ((part ? p + u * kSlots : p) * a.m + i) * 2);
        if (!part) v[u] = f32x2{-__builtin_inff(), 0.0f};
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) join_stats(&top, &sum, v[u][0], v[u][1]);
    }
  }
  tops[slot][c] = top;
  sums[slot][c] = sum;
  __syncthreads();
  // the slots' in two steps: eight by eight, then those
  if (slot < 8 && there) {
    top = tops[slot * 8][c];
    sum = sums[slot * 8][c];
    for (int s = 1; s < 8; ++s) join_stats(&top, &sum, tops[slot * 8 + s][c], sums[slot * 8 + s][c]);
  }
  __syncthreads();
  if (slot < 8) {
    tops[slot][c] = top;
    sums[slot][c] = sum;
  }
  __syncthreads();
  if (slot == 0 && there) {
    for (int s = 1; s < 8; ++s) join_stats(&top, &sum, tops[s][c], sums[s][c]);
    if (a.run && !a.first) join_stats(&top, &sum, a.run[i * 2], a.run[i * 2 + 1]);
    if (a.run && !a.last) {
      a.run[i * 2] = top;
      a.run[i * 2 + 1] = sum;
    }
    norms[c] = top + logf(sum);
  }
  if (!a.last) return;
  __syncthreads();
  const float lse = there ? norms[c] : 0.0f;
  if (a.weights) {
    float s = 0.0f;
    if (there) {
      for (int e = slot; e < a.list.per_row; e += kSlots) {
        const float w = a.weights[i * a.list.per_row + e];
        if (w != 0.0f) s += w * (logf(w) - a.listed[i * a.list.per_row + e] + lse);
      }
    }
    terms[slot][c] = s;
    __syncthreads();
    if (slot != 0 || !there) return;
    for (int q = 1; q < kSlots; ++q) s += terms[q][c];
    a.loss[i] = s;
  } else {
    if (slot != 0 || !there) return;
    const int64_t y = class_at(a.list, i, 0);
    a.loss[i] = y < 0 ? 0.0f : y < a.n ? lse - a.listed[i] : __builtin_nanf("");
  }
  a.lse[i] = lse;
}

// A workgroup of kRowThreads a row: each thread keeps the largest t and the sum of its classes, those join through LDS. (Statistics
// and loss in launches of their own took 3 us more of 13 rows.)
template <int kRowThreads>
__global__ __launch_bounds__(kRowThreads) void loss_few_rows(LossForwardArgs a, LossFinishArgs f) {
  constexpr int kRowWaves = kRowThreads / 64;
  __shared__ float tops[kRowWaves], sums[kRowWaves], terms[kRowWaves];
  __shared__ uint8_t places[256];
  constexpr int kQuads = 4;
  const int64_t i = blockIdx.x, n = a.product.n;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (f.teacher.teacher && wave == 0) teacher_row(f.teacher, i, places);
  float top = -__builtin_inff(), sum = 0.0f;
  for (int64_t j0 = threadIdx.x * 4; j0 < n; j0 += kQuads * 4 * kRowThreads) {
    f32x4 t[kQuads];
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
      const int64_t j = j0 + q * 4 * kRowThreads;
      t[q] = few_logits(a, i, j, n - j >= 4 ? 4 : (int)(n > j ? n - j : 0));
    }
    float largest = t[0][0];
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) largest = fmaxf(largest, t[q][e]);
    const float from = largest == -__builtin_inff() ? 0.0f : largest;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) s += fast_exp(t[q][e] - from);
    join_stats(&top, &sum, largest, s);
  }
  const float wave_top = wave_max(top), from = wave_top == -__builtin_inff() ? 0.0f : wave_top;
  sum = group_sum(sum * fast_exp(top - from), 64);
  if (lane == 0) {
    tops[wave] = wave_top;
    sums[wave] = sum;
  }
  __syncthreads();
  top = tops[0];
  sum = sums[0];
  for (int w = 1; w < kRowWaves; ++w) join_stats(&top, &sum, tops[w], sums[w]);
  const float lse = top + logf(sum);
  float loss = 0.0f;
  if (f.weights) {
    for (int e = threadIdx.x; e < f.list.per_row; e += kRowThreads) {
      const float w = f.weights[i * f.list.per_row + e];
      const int64_t c = class_at(f.list, i, e);
      if (w != 0.0f) loss += w * (logf(w) - (c >= 0 && c < n ? few_logits(a, i, c, 1)[0] : 0.0f) + lse);
    }
    loss = group_sum(loss, 64);
    if (lane == 0) terms[wave] = loss;
    __syncthreads();
    loss = terms[0];
    for (int w = 1; w < kRowWaves; ++w) loss += terms[w];
  } else if (threadIdx.x == 0) {
    const int64_t y = class_at(f.list, i, 0);
    loss = y < 0 ? 0.0f : y < n ? lse - few_logits(a, i, y, 1)[0] : __builtin_nanf("");
  }
  if (threadIdx.x != 0) return;
  f.loss[i] = loss;
  f.lse[i] = lse;
}

// A workgroup takes 1024 columns of kMemoryRows rows, four a thread. What their lists take off d is summed in LDS first: one
// entry a thread at a time. (Each thread looking through the lists of its rows took 1.4 us a place of 300 rows.)
template <typename T>
__global__ __launch_bounds__(256) void loss_gradient_memory(LossGradientArgs a) {
  __shared__ f32x4 targets[kMemoryRows][256];
  const ProductArgs& p = a.product;
  const int64_t j0 = (int64_t)blockIdx.x * 1024, j = j0 + threadIdx.x * 4, i0 = (int64_t)blockIdx.y * kMemoryRows;
  const int rows = p.m - i0 < kMemoryRows ? (int)(p.m - i0) : (int)kMemoryRows;
  const int count = p.n - j >= 4 ? 4 : p.n > j ? (int)(p.n - j) : 0;
#pragma unroll
  for (int r = 0; r < kMemoryRows; ++r) targets[r][threadIdx.x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  constexpr int kBatch = 4;
  const int per_row = a.list.per_row, total = rows * per_row;
  for (int at0 = threadIdx.x; at0 < total; at0 += kBatch * 256) {
    int64_t c[kBatch];
    int row[kBatch], e[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at = at0 + b * 256 < total ? at0 + b * 256 : at0;
      row[b] = at / per_row;
      e[b] = at - row[b] * per_row;
      c[b] = class_at(a.list, i0 + row[b], e[b]) - j0;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (at0 + b * 256 >= total || c[b] < 0 || c[b] >= 1024 || c[b] >= p.n - j0) continue;
      const float factor = a.factor[i0 + row[b]], w = a.weights ? a.weights[(i0 + row[b]) * per_row + e[b]] : 1.0f;
      if (factor != 0.0f && w != 0.0f)
        __hip_atomic_fetch_add(reinterpret_cast<float*>(&targets[row[b]][0]) + c[b], factor * w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  }
  __syncthreads();
  if (j >= a.ldd) return;
  constexpr bool kScaled = sizeof(T) == 2;
  const float scale = kScaled && a.scale ? *a.scale : 1.0f;
  f32x4 bias = {0.0f, 0.0f, 0.0f, 0.0f}, sum = bias;
  if (a.bias && count > 0) bias = load4<float>(a.bias + j, count) * a.inv_temperature;
#pragma unroll 2
  for (int r = 0; r < rows; ++r) {
    const int64_t i = i0 + r;
    const float factor = a.factor[i], lse = a.lse[i];
    f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
    if (factor != 0.0f && count > 0) {
      const f32x4 z = load4<float>(p.partial + i * p.n + j, count), target = targets[r][threadIdx.x];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = e < count ? factor * fast_exp(fmaf(z[e], a.inv_temperature, bias[e]) - lse) - target[e] : 0.0f;
    }
    sum += d;
    if (a.d) {
      typename Vec<T>::x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = (T)(kScaled ? d[e] * scale : d[e]);
      *reinterpret_cast<typename Vec<T>::x4*>(static_cast<T*>(a.d) + i * a.ldd + j) = o;
    }
  }
  if (a.sums && count > 0) store4<float>(a.sums + (int64_t)blockIdx.y * p.n + j, sum, count);
}

// Weights of rows of more classes, a workgroup a row. A class finds the places that list it through a table in LDS, at most
// half full: its least place and their number; where there are several, the first adds them in their order. (Comparing every
// two places took 1032 us of 300 rows of 1000, 72 of 256 a row.)
constexpr int kPlaces = 2 * kMostListed;

__global__ __launch_bounds__(256) void teacher_weights(TeacherArgs a) {
  __shared__ int32_t keys[kPlaces];
  __shared__ uint32_t least[kPlaces], many[kPlaces];
  __shared__ float weights[kMostListed];
  __shared__ uint16_t places[kMostListed];
  __shared__ float tops[4], sums[4];
  __shared__ int bads[4];
  constexpr int kEach = kMostListed / 256;
  const int64_t i = blockIdx.x;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, count = a.list.per_row;
  for (int h = threadIdx.x; h < kPlaces; h += 256) {
    keys[h] = -1;
    least[h] = ~0u;
    many[h] = 0;
  }
  __syncthreads();
  float t[kEach], top = -__builtin_inff(), sum = 0.0f;
  bool bad = false, valid[kEach];
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    const int e = q * 256 + threadIdx.x;
    const int64_t c = e < count ? class_at(a.list, i, e) : -1;
    valid[q] = c >= 0 && c < a.n;
    t[q] = valid[q] ? teacher_at(a, i * a.ldt + e) * a.inv_temperature : -__builtin_inff();
    bad |= c >= a.n || t[q] != t[q];
    top = fmaxf(top, t[q]);
    if (e >= count) continue;
    uint32_t h = kPlaces;  // no place
    if (valid[q]) {
      h = (uint32_t)c * 2654435761u >> 21;
      static_assert(kPlaces == 1 << 11, "bits of a place");
      for (int old; (old = atomicCAS(&keys[h], -1, (int32_t)c)) != -1 && old != (int32_t)c;) h = (h + 1) % kPlaces;
      atomicMin(&least[h], (uint32_t)e);
      atomicAdd(&many[h], 1u);
    }
    places[e] = (uint16_t)h;
  }
  top = wave_max(top);
  bad = __any(bad);
  if (lane == 0) {
    tops[wave] = top;
    bads[wave] = bad;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    top = fmaxf(top, tops[w]);
    bad |= bads[w] != 0;
  }
  const float from = top == -__builtin_inff() ? 0.0f : top;
  float own[kEach];
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    const int e = q * 256 + threadIdx.x;
    own[q] = expf(t[q] - from);
    if (e < count) weights[e] = own[q];
    sum += own[q];
  }
  sum = group_sum(sum, 64);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  sum = sums[0] + sums[1] + sums[2] + sums[3];
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    const int e = q * 256 + threadIdx.x;
    if (e >= count) continue;
    float w = 0.0f;
    if (valid[q] && least[places[e]] == (uint32_t)e) {
      w = own[q];
      if (many[places[e]] > 1)
        for (int f = e + 1; f < count; ++f)
          if (places[f] == places[e]) w += weights[f];
    }
    a.weights[i * count + e] = stored_weight(bad, sum, sum > 0.0f ? w / sum : 0.0f);
  }
}

// Of a row's weights only whether there are any, and whether they are a distribution. kLanes lanes a row.
template <int kLanes>
__device__ __forceinline__ float factor_of(const LossFactorArgs& a, int64_t i) {
  if (a.weights) {
    bool any = false, bad = false;
#pragma unroll 8
    for (int e = threadIdx.x % kLanes; e < a.list.per_row; e += kLanes) {
      const float w = a.weights[i * a.list.per_row + e];
      any |= w != 0.0f;
      bad |= w != w;
    }
    if constexpr (kLanes > 1) {
      const int shift = (threadIdx.x & 63) / kLanes * kLanes;
      const uint64_t lanes = ~(uint64_t)0 >> (64 - kLanes);
      any = (__ballot(any) >> shift & lanes) != 0;
      bad = (__ballot(bad) >> shift & lanes) != 0;
    }
    return bad ? __builtin_nanf("") : any ? a.grad[i] * a.inv_temperature : 0.0f;
  }
  const int64_t y = class_at(a.list, i, 0);
  return y < 0 ? 0.0f : y < a.n ? a.grad[i] : __builtin_nanf("");
}

template <int kLanes>
__global__ __launch_bounds__(256) void loss_factor(LossFactorArgs a) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kLanes;
  const float f = factor_of<kLanes>(a, i < a.m ? i : a.m - 1);
  if (i < a.m && threadIdx.x % kLanes == 0) a.factor[i] = f;
}

// The scale, in one workgroup; kFactor: after forming the factors itself.
template <bool kFactor>
__global__ __launch_bounds__(1024) void loss_scale(LossFactorArgs a) {
  __shared__ float lds[16];
  float top = 0.0f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.m; i += 1024) {
    float f;
    if (kFactor) a.factor[i] = f = factor_of<1>(a, i);
    else f = a.factor[i];
    f = fabsf(f);
    top = f < __builtin_inff() ? fmaxf(top, f) : top;
  }
#pragma unroll
  for (int by = 1; by < 64; by *= 2) top = fmaxf(top, __shfl_xor(top, by));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) top = fmaxf(top, lds[w]);
  if (top == 0.0f) top = 1.0f;
  const int e = ilogbf(top), up = 13 - e > 120 ? 120 : 13 - e < -120 ? -120 : 13 - e;
  const float digits = ldexpf(top, -e);
  a.scale[0] = ldexpf(1.0f / digits, up);
  a.scale[1] = ldexpf(digits, -up);
}

__global__ __launch_bounds__(256) void sum_slices(float* slices, int64_t count, int64_t quads) {
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < quads; q += (int64_t)gridDim.x * 256) {
    f32x4* p = reinterpret_cast<f32x4*>(slices) + q;
    f32x4 s = p[0];
#pragma unroll 4
    for (int64_t c = 1; c < count; ++c) s += p[c * quads];
    p[0] = s;
  }
}

template <typename T>
void forward_type(const LossForwardArgs& a, hipStream_t s) {
  const uint32_t groups = (uint32_t)a.product.tiles();
  if constexpr (sizeof(T) == 2) {
    if (a.product.tile == 256) {
      loss_forward<T, 256><<<groups, kThreads, 0, s>>>(a);
      return;
    }
  }
  if (a.product.tile == 128) loss_forward<T, 128><<<groups, kThreads, 0, s>>>(a);
  else loss_forward<T, 64><<<groups, kThreads, 0, s>>>(a);
}

template <typename T>
void gradient_type(const LossGradientArgs& a, hipStream_t s) {
  const uint32_t groups = (uint32_t)a.product.tiles();
  if constexpr (sizeof(T) == 2) {
    if (a.product.tile == 256) {
      loss_gradient<T, 256><<<groups, kThreads, 0, s>>>(a);
      return;
    }
  }
  if (a.product.tile == 128) loss_gradient<T, 128><<<groups, kThreads, 0, s>>>(a);
  else loss_gradient<T, 64><<<groups, kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_loss_forward(const LossForwardArgs& a, hipStream_t s) {
  if (a.product.type == kBf16) forward_type<__bf16>(a, s);
  else if (a.product.type == kF16) forward_type<_Float16>(a, s);
  else forward_type<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_loss_gradient(const LossGradientArgs& a, hipStream_t s) {
  if (a.product.type == kBf16) gradient_type<__bf16>(a, s);
  else if (a.product.type == kF16) gradient_type<_Float16>(a, s);
  else gradient_type<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_loss_few(const LossForwardArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.product.n + kFewChunk - 1) / kFewChunk), (unsigned)a.product.m);
  loss_few<<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_loss_few_rows(const LossForwardArgs& a, const LossFinishArgs& f, hipStream_t s) {
  if (a.product.n > 4096) loss_few_rows<1024><<<(unsigned)a.product.m, 1024, 0, s>>>(a, f);
  else if (a.product.n > 256) loss_few_rows<256><<<(unsigned)a.product.m, 256, 0, s>>>(a, f);
  else loss_few_rows<64><<<(unsigned)a.product.m, 64, 0, s>>>(a, f);
  return hipGetLastError();
}

hipError_t launch_loss_gradient_memory(const LossGradientArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.ldd / 4 + 255) / 256), (unsigned)((a.product.m + kMemoryRows - 1) / kMemoryRows));
  if (a.product.type == kBf16) loss_gradient_memory<__bf16><<<grid, 256, 0, s>>>(a);
  else if (a.product.type == kF16) loss_gradient_memory<_Float16><<<grid, 256, 0, s>>>(a);
  else loss_gradient_memory<float><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_list_order(const OrderArgs& a, hipStream_t s) {
  list_order<<<(unsigned)((a.m + a.order.strip_rows - 1) / a.order.strip_rows), kOrderThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_loss_finish(const LossFinishArgs& a, hipStream_t s) {
  loss_finish<<<(unsigned)((a.m + 15) / 16), 16 * kSlots, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_sum_slices(float* slices, int64_t count, int64_t elements, hipStream_t s) {
  const int64_t groups = (elements / 4 + 255) / 256;
  sum_slices<<<(unsigned)(groups < 65536 ? groups : 65536), 256, 0, s>>>(slices, count, elements / 4);
  return hipGetLastError();
}

hipError_t launch_teacher_weights(const TeacherArgs& a, hipStream_t s) {
  if (a.m == 0 || a.list.per_row == 0) return hipSuccess;
  teacher_weights<<<(unsigned)a.m, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_loss_factor(const LossFactorArgs& a, hipStream_t s) {
  // two launches: 11 us of 200 rows, one: 2.4; at 2047 x 32 one takes 12.7
  if (a.scale && a.list.per_row <= 32 && a.m * a.list.per_row <= 8192) {
    loss_scale<true><<<1, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const auto groups = [&](int lanes) { return (unsigned)((a.m * lanes + 255) / 256); };
  // us, with 1, 16 and 64 lanes a row (500 x 512 x 2000 with its gradient): 8 weights 37.9, 38.2, 37.8; 32 47.3, 46.8, 46.8;
  // 300 87, 72, 73; 1000 184, 138, 137
  if (!a.weights || a.list.per_row <= 8) loss_factor<1><<<groups(1), 256, 0, s>>>(a);
  else loss_factor<16><<<groups(16), 256, 0, s>>>(a);
  if (a.scale) loss_scale<false><<<1, 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace xtvxy
