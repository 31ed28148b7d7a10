// Products of any size, alignment and element type in 64 x 64 tiles, for small or ragged layers and small
// fp32 gradients, and the kernels around a product: the slope of the activation with its column sums,
// copies with padded rows, and the sum of a split contraction's parts.
//
// These are bound by latency: a launch, the first loads, a step's barrier and the end of the tile. fp16
// 1023 x 1111 x 777 (35 steps) takes 13.8 us, the slope of 4096 x 4096 in bf16 21 us (4.8 TB/s), of
// 1501 x 501 5.
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

  __device__ __forceinline__ void load(const T* base, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t k_end) {
    const int t = threadIdx.x;
    const int64_t row = kContractionMajor ? r0 + (t & 7) * 8 : r0 + (t >> 2);
    const int64_t k = kContractionMajor ? k0 + (t >> 3) : k0 + (t & 3) * 8;
    const int64_t outer = kContractionMajor ? k : row, inner = kContractionMajor ? row : k;
    const int64_t outer_end = kContractionMajor ? k_end : rows, inner_end = kContractionMajor ? rows : k_end;
    const int64_t left = outer < outer_end ? inner_end - inner : 0;
    const T* p = base + outer * ld + inner;
    if (left >= 8) {  // memory takes unaligned accesses
      __builtin_memcpy(&v, p, sizeof(v));
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

// d = g act'(z) of 8 elements in fp32.
template <typename V>
__device__ __forceinline__ f32x8 slope8(V g, V z, int act) {
  f32x8 d;
#pragma unroll
  for (int c = 0; c < 8; ++c) d[c] = (float)g[c];
  switch (act) {
#define XTVXY_SLOPE_CASE(A)                                                                  \
  case A:                                                                                    \
    _Pragma("unroll") for (int c = 0; c < 8; ++c) d[c] *= slope<A>((float)z[c]);             \
    break;
    XTVXY_SLOPE_CASE(XTVXY_ACT_RELU)
    XTVXY_SLOPE_CASE(XTVXY_ACT_GELU)
    XTVXY_SLOPE_CASE(XTVXY_ACT_GELU_TANH)
    XTVXY_SLOPE_CASE(XTVXY_ACT_SILU)
#undef XTVXY_SLOPE_CASE
    default: break;
  }
  return d;
}

// A 64 x 64 tile of C, four wavefronts of 32 x 32 each. The product is formed transposed (B's rows as
// the matrix instruction's first operand), so that a lane ends with four neighbouring columns of one
// row of C. The next step's elements are in flight while the present one's products run. The first operand
// is G, and d is formed between its load and its store to LDS, in the element type (as slope_rows does); where the contraction runs over d's rows
// and this is the product's first tile column, its column sums are taken from the unrounded d on the way.
template <typename T, bool kAMajor, bool kBMajor>
__device__ __forceinline__ void tile(const ProductArgs& a, uint32_t id, const GradientArgs* grad, T* sa, T* sb) {
  typedef typename Vec<T>::x8 frag;
  const uint32_t tiles_n = (uint32_t)((a.n + kTile - 1) / kTile), tiles = (uint32_t)((a.m + kTile - 1) / kTile) * tiles_n;
  const uint32_t split = id / tiles, t = id % tiles;
  const int64_t i0 = (int64_t)(t / tiles_n) * kTile, j0 = (int64_t)(t % tiles_n) * kTile;
  const int64_t k0 = (int64_t)split * a.k_per_split;
  const int64_t k_end = k0 + a.k_per_split < a.k ? k0 + a.k_per_split : a.k;
  const T* A = static_cast<const T*>(a.A);
  const T* B = static_cast<const T*>(a.B);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
  const int r = lane & 15, g = lane >> 4;
  const bool with_pre = grad->pre, with_sums = kAMajor && grad->own_sums && j0 == 0;

  f32x4 acc[2][2] = {};
  f32x8 sum = {};
  TileLoad<T, kAMajor> la, lz;
  TileLoad<T, kBMajor> lb;
  const auto load = [&](int64_t k) {
    la.load(A, a.lda, i0, a.m, k, k_end);
    if (with_pre) lz.load(static_cast<const T*>(grad->pre), grad->ldp, i0, a.m, k, k_end);
    lb.load(B, a.ldb, j0, a.n, k, k_end);
  };
  load(k0);
  for (int64_t k = k0; k < k_end; k += kTileDepth) {
    const f32x8 d = slope8(la.v, lz.v, with_pre ? grad->act : XTVXY_ACT_NONE);
    if (with_sums) sum += d;
#pragma unroll
    for (int c = 0; c < 8; ++c) la.v[c] = (T)d[c];
    la.store(sa);
    lb.store(sb);
    __syncthreads();
    if (k + kTileDepth < k_end) load(k + kTileDepth);
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
        float* p = a.partial + ((int64_t)split * a.m + i) * a.n + j;
        store4<float>(p, acc[x][y], a.n - j >= 4 ? 4 : (int)(a.n - j));
      } else {
        epilogue4<T>(a.e, i, j, a.n, acc[x][y]);
      }
    }
  if (with_sums) {
    // thread t holds columns 8 (t & 7) + 0..7 of every depth's step t >> 3
    float* part = reinterpret_cast<float*>(sa);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float s = sum[c];
      s += __shfl_xor(s, 8);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (lane < 8) part[wave * 64 + lane * 8 + c] = s;
    }
    __syncthreads();
    const int64_t i = i0 + threadIdx.x;
    if (threadIdx.x < 64 && i < a.m)
      grad->own_sums[(int64_t)split * a.m + i] =
          part[threadIdx.x] + part[64 + threadIdx.x] + part[128 + threadIdx.x] + part[192 + threadIdx.x];
  }
}

// The layer's tile for rows of any length and alignment: the same 64 x 64 outputs by four wavefronts, with
// four steps of both operands in flight in registers and two LDS buffers, so that a step has one barrier.
// A row's end needs no branch: its last 8 elements are loaded as they lie and shifted so that zeros stand
// beyond the end; rows that do not exist are loaded as the last one and not stored. kShort: rows of fewer
// than 8 elements, loaded one by one (in a kernel of its own: a branch makes every load wait). An XCD takes
// neighbouring tiles, whose operands its L2 then holds (fp16 4000 x 2001 x 4000: 256 us in launch order, 80 so).
template <typename T, bool kShort>
__global__ __launch_bounds__(kThreads) void layer_tile(ProductArgs a) {
  typedef typename Vec<T>::x8 frag;
  constexpr int kAhead = 4, kBuffer = 2 * kTile * kPitch;
  __shared__ __align__(16) T lds[2 * kBuffer];
  const uint32_t tiles_n = (uint32_t)((a.n + kTile - 1) / kTile), tiles = (uint32_t)((a.m + kTile - 1) / kTile) * tiles_n;
  const uint32_t split = blockIdx.x / tiles, t = spread(blockIdx.x % tiles, tiles);
  const int64_t i0 = (int64_t)(t / tiles_n) * kTile, j0 = (int64_t)(t % tiles_n) * kTile;
  const int64_t k0 = (int64_t)split * a.k_per_split;
  const int64_t k_end = k0 + a.k_per_split < a.k ? k0 + a.k_per_split : a.k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32, r = lane & 15, g = lane >> 4;
  const int row = threadIdx.x >> 2, chunk = (threadIdx.x & 3) * 8;
  const T* pa = static_cast<const T*>(a.A) + (i0 + row < a.m ? i0 + row : a.m - 1) * a.lda;
  const T* pb = static_cast<const T*>(a.B) + (j0 + row < a.n ? j0 + row : a.n - 1) * a.ldb;
  frag va[kAhead], vb[kAhead];
  const auto load = [&](frag& v, const T* p, int64_t k) {
    k += chunk;
    if (!kShort) {
      __builtin_memcpy(&v, p + (k <= k_end - 8 ? k : k_end - 8), sizeof(v));  // memory takes unaligned accesses
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < k_end ? p[k + i] : (T)0.0f;
    }
  };
  const auto trim = [&](frag& v, int64_t k) {
    const int64_t over = k + chunk + 8 - k_end;  // elements beyond the end
    if (kShort) return;
    const int shift = over <= 0 ? 0 : over < 8 ? (int)over : 8;
#pragma unroll
    for (int by = 8; by > 0; by /= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = shift & by ? (i + by < 8 ? v[(i + by) & 7] : (T)0.0f) : v[i];
  };
  // Steps in fours without a branch around a load: where its number is not known the compiler waits for
  // all of them. Steps beyond the end load the row's last elements again and multiply zeros.
  if (k0 < k_end) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      load(va[u], pa, k0 + u * kTileDepth);
      load(vb[u], pb, k0 + u * kTileDepth);
    }
  }
  f32x4 acc[2][2] = {};
  for (int64_t k4 = k0; k4 < k_end; k4 += kAhead * kTileDepth) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t k = k4 + u * kTileDepth;
      if (k + kTileDepth > k_end) {
        trim(va[u], k);
        trim(vb[u], k);
      }
      T* sa = lds + (u & 1) * kBuffer;
      T* sb = sa + kTile * kPitch;
      *reinterpret_cast<frag*>(sa + row * kPitch + chunk) = va[u];
      *reinterpret_cast<frag*>(sb + row * kPitch + chunk) = vb[u];
      __syncthreads();  // the buffer's last readers have passed the barrier of the step between
      load(va[u], pa, k + kAhead * kTileDepth);
      load(vb[u], pb, k + kAhead * kTileDepth);
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
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int64_t i = i0 + wi + x * 16 + r, j = j0 + wj + y * 16 + g * 4;
      if (i >= a.m || j >= a.n) continue;
      if (a.splits > 1) store4<float>(a.partial + ((int64_t)split * a.m + i) * a.n + j, acc[x][y], a.n - j >= 4 ? 4 : (int)(a.n - j));
      else epilogue4<T>(a.e, i, j, a.n, acc[x][y]);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gradient_tile(GradientArgs a) {
  __shared__ __align__(16) T sa[kTile * kPitch], sb[kTile * kPitch];
  if (blockIdx.x < a.dx_groups) tile<T, false, true>(a.dx, blockIdx.x, &a, sa, sb);
  else tile<T, true, true>(a.dw, blockIdx.x - a.dx_groups, &a, sa, sb);
}

// Four neighbouring outputs of a split product by four neighbouring lanes: each sums every fourth part
// in ascending order (its loads are under way together), the lanes' sums join in a fixed order.
template <typename T>
__device__ __forceinline__ void finish_quad(const ProductArgs& a, int64_t at) {
  const int part = (int)(at & 3);
  int64_t q = at >> 2, i, j, stride;
  const float* p = a.partial;
  if (a.tile) {  // split tiles in areas of their own
    const int edge = 31 - __builtin_clz(a.tile), r = (int)(q >> (2 * edge - 2));
    const int row = (int)(q >> (edge - 2)) & (a.tile - 1), quad = (int)q & (a.tile / 4 - 1);
    const uint32_t rest = (uint32_t)(a.tiles() - a.whole);
    int64_t tm, tn;
    tile_of(a, (uint32_t)a.whole + spread((uint32_t)r, rest), &tm, &tn);
    i = tm * a.tile + row;
    j = tn * a.tile + quad * 4;
    p += q * 4;
    stride = (int64_t)rest << (2 * edge);
  } else {
    const int64_t quads = (a.n + 3) / 4;
    i = q / quads;
    j = (q - i * quads) * 4;
    p += i * a.n + j;
    stride = a.m * a.n;
  }
  const bool exists = i < a.m && j < a.n;
  const int count = a.n - j >= 4 ? 4 : (int)(a.n - j);
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  if (exists) {
#pragma unroll 4
    for (int s = part; s < a.splits; s += 4) z += load4<float>(p + s * stride, count);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    z[c] += __shfl_xor(z[c], 1);
    z[c] += __shfl_xor(z[c], 2);
  }
  if (exists && part == 0) epilogue4<T>(a.e, i, j, a.n, z);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void product_finish(ProductArgs a) {
  finish_quad<T>(a, (int64_t)blockIdx.x * kThreads + threadIdx.x);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gradient_finish(GradientArgs a) {
  __shared__ double lds[16 * kSumColumns];
  uint32_t id = blockIdx.x;
  if (id < a.dx_groups) return finish_quad<T>(a.dx, (int64_t)id * kThreads + threadIdx.x);
  id -= a.dx_groups;
  if (id < a.dw_groups) return finish_quad<T>(a.dw, (int64_t)id * kThreads + threadIdx.x);
  column_sum(a.sums, a.sum_rows, a.n, a.db, id - a.dw_groups, lds);
}

// d = g act'(pre) in fp32, stored in the element type, which is what the products' instructions take; the
// column sums db take d before that rounding. It makes the error of 16-bit dX and dW 1.41 times what rounding
// them alone costs (bf16 2.35e-3 against 1.66e-3 in the 2-norm, fp16 2.94e-4 against 2.08e-4); d as the sum of
// two 16-bit parts would take twice the products.
// A workgroup walks rows_per_group rows of 8 kLanes columns, a thread owns 8 neighbouring columns of
// every 256 / kLanes-th row.
template <typename T, int kAct, int kLanes>
__global__ __launch_bounds__(kThreads) void slope_rows(SlopeArgs a) {
  constexpr int kSlots = kThreads / kLanes;  // rows at once
  const int slot = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t j = ((int64_t)blockIdx.x * kLanes + lane) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * a.rows_per_group;
  const int64_t r1 = r0 + a.rows_per_group < a.m ? r0 + a.rows_per_group : a.m;
  const T* G = static_cast<const T*>(a.g);
  const T* P = static_cast<const T*>(a.pre);
  T* D = static_cast<T*>(a.d);
  typedef typename Vec<T>::x8 v8;
  float sum[8] = {};
  const int count = a.n - j >= 8 ? 8 : (a.n > j ? (int)(a.n - j) : 0);
  // The lane of a row's last, partial eight loads the eight that end with the row and shifts: a branch
  // around its loads would make every row wait for them (1501 x 501: 13.8 us against 5).
  const int shift = a.n >= 8 ? 8 - count : 0;
  const bool shifts = __any(count > 0 && shift > 0);
  const T* Gj = G + j - shift;
  const T* Pj = P + j - shift;
  if (count > 0) {
#pragma unroll 4
    for (int64_t i = r0 + slot; i < r1; i += kSlots) {
      v8 g = {}, z = {}, o;
      if (a.n >= 8) {  // memory takes unaligned accesses
        __builtin_memcpy(&g, Gj + i * a.ldg, sizeof(g));
        if (kAct != XTVXY_ACT_NONE) __builtin_memcpy(&z, Pj + i * a.ldp, sizeof(z));
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < count) {
            g[c] = Gj[i * a.ldg + c];
            if (kAct != XTVXY_ACT_NONE) z[c] = Pj[i * a.ldp + c];
          }
      }
      float x[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[c] = (float)g[c];
        if (kAct != XTVXY_ACT_NONE) x[c] *= slope<kAct>((float)z[c]);
      }
      if (shifts) {  // zeros come in from the right
#pragma unroll
        for (int by = 4; by > 0; by /= 2)
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] = shift & by ? (c + by < 8 ? x[c + by] : 0.0f) : x[c];
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = (T)x[c];
      if (D) *reinterpret_cast<v8*>(D + i * a.ldd + j) = o;  // ldd is a multiple of 8; missing columns are zero
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += x[c];
    }
  }
  if (!a.sums) return;
  // the row slots' sums: within a wavefront by lane exchanges, then through LDS
  __shared__ float part[kThreads / 64][kLanes < 64 ? kLanes : 64][9];
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
#pragma unroll
    for (int d = kLanes; d < 64; d *= 2) sum[c] += __shfl_xor(sum[c], d);
    if ((threadIdx.x & 63) < kLanes) part[wave][lane][c] = sum[c];
  }
  __syncthreads();
  if (threadIdx.x >= kLanes || count == 0) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float s = part[0][lane][c];
    for (int p = 1; p < kThreads / 64; ++p) s += part[p][lane][c];
    if (c < count) a.sums[(int64_t)blockIdx.y * a.n + j + c] = s;
  }
}

// 16 bytes of a row at a time; the source may have any alignment (memory takes unaligned accesses).
// Positions are 32-bit where they fit: two 64-bit divisions cost as much as the copy of a chunk.
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_rows(PackArgs a) {
  constexpr int kChunk = 16 / sizeof(T);
  typedef T chunk __attribute__((ext_vector_type(kChunk)));
  const PackJob& job = a.job[blockIdx.y];
  const int64_t chunks = job.ldd / kChunk, total = job.rows * chunks;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < total; at += (int64_t)gridDim.x * kThreads) {
    const bool fits = total <= INT32_MAX;
    const int64_t i = fits ? (uint32_t)at / (uint32_t)chunks : at / chunks, c = (at - i * chunks) * kChunk;
    const T* p = static_cast<const T*>(job.src) + i * job.ld + c;
    const int64_t left = job.cols - c;
    T x[kChunk];
    load_elems<T, kChunk>(p, left >= kChunk ? kChunk : (int)left, x);
    chunk v;
#pragma unroll
    for (int e = 0; e < kChunk; ++e) v[e] = x[e];
    *reinterpret_cast<chunk*>(static_cast<T*>(job.dst) + i * job.ldd + c) = v;
  }
}

template <typename T, int kLanes>
hipError_t slope_lanes(const SlopeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 8 * kLanes - 1) / (8 * kLanes)), (unsigned)a.groups);
  switch (a.pre ? a.act : XTVXY_ACT_NONE) {
    case XTVXY_ACT_RELU: slope_rows<T, XTVXY_ACT_RELU, kLanes><<<grid, kThreads, 0, s>>>(a); break;
    case XTVXY_ACT_GELU: slope_rows<T, XTVXY_ACT_GELU, kLanes><<<grid, kThreads, 0, s>>>(a); break;
    case XTVXY_ACT_GELU_TANH: slope_rows<T, XTVXY_ACT_GELU_TANH, kLanes><<<grid, kThreads, 0, s>>>(a); break;
    case XTVXY_ACT_SILU: slope_rows<T, XTVXY_ACT_SILU, kLanes><<<grid, kThreads, 0, s>>>(a); break;
    default: slope_rows<T, XTVXY_ACT_NONE, kLanes><<<grid, kThreads, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

// A row's lanes: as many as it has groups of 8 columns, so that narrow layers' rows share a wavefront.
template <typename T>
hipError_t slope_for(const SlopeArgs& a, hipStream_t s) {
  return a.n > kSlopeNarrow ? slope_lanes<T, 64>(a, s) : slope_lanes<T, 16>(a, s);
}

uint32_t tile_groups(const ProductArgs& a) {
  return (uint32_t)(((a.m + kTile - 1) / kTile) * ((a.n + kTile - 1) / kTile) * a.splits);
}

template <typename T>
void layer_tile_for(const ProductArgs& a, hipStream_t s) {
  if (a.k < 8) layer_tile<T, true><<<tile_groups(a), kThreads, 0, s>>>(a);
  else layer_tile<T, false><<<tile_groups(a), kThreads, 0, s>>>(a);
}

}  // namespace

uint32_t quad_groups(const ProductArgs& a) {
  const int64_t quads = a.tile ? (a.tiles() - a.whole) * a.tile * (a.tile / 4) : a.m * ((a.n + 3) / 4);
  return (uint32_t)((quads * 4 + kThreads - 1) / kThreads);
}

hipError_t launch_layer_tile(const ProductArgs& a, hipStream_t s) {
  if (a.type == kBf16) layer_tile_for<__bf16>(a, s);
  else if (a.type == kF16) layer_tile_for<_Float16>(a, s);
  else layer_tile_for<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_gradient_tile(const GradientArgs& args, int type, hipStream_t s) {
  GradientArgs a = args;
  a.dx_groups = a.dx.m > 0 ? tile_groups(a.dx) : 0;
  a.dw_groups = a.dw.m > 0 ? tile_groups(a.dw) : 0;
  const uint32_t grid = a.dx_groups + a.dw_groups;
  if (grid == 0) return hipSuccess;
  if (type == kBf16) gradient_tile<__bf16><<<grid, kThreads, 0, s>>>(a);
  else if (type == kF16) gradient_tile<_Float16><<<grid, kThreads, 0, s>>>(a);
  else gradient_tile<float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_product_finish(const ProductArgs& a, hipStream_t s) {
  if (a.type == kBf16) product_finish<__bf16><<<quad_groups(a), kThreads, 0, s>>>(a);
  else if (a.type == kF16) product_finish<_Float16><<<quad_groups(a), kThreads, 0, s>>>(a);
  else product_finish<float><<<quad_groups(a), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_gradient_finish(const GradientArgs& args, int type, hipStream_t s) {
  GradientArgs a = args;
  a.dx_groups = a.dx.m > 0 && a.dx.splits > 1 ? quad_groups(a.dx) : 0;
  a.dw_groups = a.dw.m > 0 && a.dw.splits > 1 ? quad_groups(a.dw) : 0;
  const uint32_t grid = a.dx_groups + a.dw_groups + (a.db ? (uint32_t)((a.n + kSumColumns - 1) / kSumColumns) : 0);
  if (grid == 0) return hipSuccess;
  if (type == kBf16) gradient_finish<__bf16><<<grid, kThreads, 0, s>>>(a);
  else if (type == kF16) gradient_finish<_Float16><<<grid, kThreads, 0, s>>>(a);
  else gradient_finish<float><<<grid, kThreads, 0, s>>>(a);
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


}  // namespace xtvxy
