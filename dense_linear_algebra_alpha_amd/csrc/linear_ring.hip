// The fully connected layer's product and its gradient's two by the large-tile ring kernel (linear_ring.h), with the
// layer's epilogue.
#include "linear_ring.h"

namespace xtvxy {
namespace {

// The epilogue of a wavefront's staged rows from (i0, j0) on, 8 columns a lane. kPlain: the sums alone.
template <typename T, int kAct, int WN, int kRows, bool kPlain>
__device__ __forceinline__ void epilogue_rows(const float* area, const ProductArgs& a, int64_t i0, int64_t j0) {
  constexpr int kLanes = WN / 8, kStep = 64 / kLanes;  // lanes of a row, rows at once
  const LinearEpilogue e = kPlain ? LinearEpilogue{nullptr, nullptr, 0, nullptr, 0, a.e.out, a.e.ldo, kAct} : a.e;
  const int lane = threadIdx.x & 63, c8 = lane % kLanes;
  const int64_t j = j0 + c8 * 8;
  const int count = a.n - j >= 8 ? 8 : (a.n > j ? (int)(a.n - j) : 0);
  if (count == 0) return;
  const float scale = kPlain && a.scale ? *a.scale : 1.0f;
  float bias[8] = {};
  if (e.bias) load_elems<float, 8>(e.bias + j, count, bias);
  const int rows = a.m - i0 >= kRows ? kRows : (int)(a.m - i0);
  const T* res = static_cast<const T*>(e.residual) + (e.residual ? i0 * e.ldr + j : 0);
  T* pre = static_cast<T*>(e.pre) + (e.pre ? i0 * e.ldp + j : 0);
  T* out = static_cast<T*>(e.out) + i0 * e.ldo + j;
  const auto run = [&](int row, int count, const T (&rv)[8]) {
    T o[8];
    const f32x8 s = staged8<WN>(area, row, c8);
    float z[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) z[c] = s[c] + bias[c];
    if (e.pre) {
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = (T)z[c];
      store_elems<T, 8>(pre + row * e.ldp, count, o);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float y = activation<sizeof(T) == 2, kAct>(z[c]);
      if (kPlain) y *= scale;
      if (e.residual) y += (float)rv[c];
      o[c] = (T)y;
    }
    store_elems<T, 8>(out + row * e.ldo, count, o);
  };
  if (count == 8) {
    // The residual of several rows is loaded before the first of them is stored (out may be the residual,
    // so the compiler keeps loads behind stores): one wait instead of one per row.
    constexpr int kBatch = kRows / kStep < 4 ? kRows / kStep : 4;
#pragma unroll 1
    for (int row = lane / kLanes; row < rows; row += kStep * kBatch) {
      T rv[kBatch][8] = {};
      if (e.residual)
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int at = row + b * kStep;
          load_elems<T, 8>(res + (at < rows ? at : row) * e.ldr, 8, rv[b]);
        }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (row + b * kStep < rows) run(row + b * kStep, 8, rv[b]);
    }
  } else {
    for (int row = lane / kLanes; row < rows; row += kStep) {
      T rv[8] = {};
      if (e.residual) load_elems<T, 8>(res + row * e.ldr, count, rv);
      run(row, count, rv);
    }
  }
}

template <typename T, int WN, int kRows>
__device__ __forceinline__ void epilogue_any(const float* area, const ProductArgs& a, int64_t i0, int64_t j0) {
  switch (a.e.act) {
    case XTVXY_ACT_RELU: epilogue_rows<T, XTVXY_ACT_RELU, WN, kRows, false>(area, a, i0, j0); break;
    case XTVXY_ACT_GELU: epilogue_rows<T, XTVXY_ACT_GELU, WN, kRows, false>(area, a, i0, j0); break;
    case XTVXY_ACT_GELU_TANH: epilogue_rows<T, XTVXY_ACT_GELU_TANH, WN, kRows, false>(area, a, i0, j0); break;
    case XTVXY_ACT_SILU: epilogue_rows<T, XTVXY_ACT_SILU, WN, kRows, false>(area, a, i0, j0); break;
    default: epilogue_rows<T, XTVXY_ACT_NONE, WN, kRows, false>(area, a, i0, j0); break;
  }
}

// The end of a tile (kPlain: of the gradient's products, which have no epilogue): its sums through LDS
// to memory. `ring` holds at least 256 (BM + BN) bytes.
template <bool kPlain>
struct StoreEnd {
  template <typename T, int BM, int BN, typename S>
  __device__ __forceinline__ void finish(const ProductArgs& a, uint8_t* ring, S& sums, const TilePlace& p) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = (wave >> 1) * (BM / 2), wj = (wave & 1) * (BN / 2);
    end_of_products(sums);
    typedef Strips<BM, BN> Strip;
    constexpr int WN = Strip::kWidth, kRows = Strip::kRows;
    float* area = reinterpret_cast<float*>(ring + wave * Strip::kArea);
#pragma unroll
    for (int part = 0; part < BM / 2 / kRows; ++part) {
      sums.template stage<WN>(area, part, kRows);
      __builtin_amdgcn_wave_barrier();
      const int i = wi + part * kRows;
      if (p.part)
        partial_rows<WN, kRows, BN>(area, p.part + i * BN + wj);
      else if (kPlain)
        epilogue_rows<T, XTVXY_ACT_NONE, WN, kRows, true>(area, a, p.i0 + i, p.j0 + wj);
      else
        epilogue_any<T, WN, kRows>(area, a, p.i0 + i, p.j0 + wj);
      __builtin_amdgcn_wave_barrier();
    }
  }
};

template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void layer_ring(ProductArgs a) {
  __shared__ __align__(1024) uint8_t ring[ring_bytes(TILE)];
  if constexpr (TILE == 256) ring_tile_halves<T, TILE, TILE, false, false>(a, blockIdx.x, ring, StoreEnd<false>());
  else ring_tile<T, TILE, TILE, false, false>(a, blockIdx.x, ring, StoreEnd<false>());
}

template <typename T, int TILE, bool kAMajor>
__device__ __forceinline__ void gradient_product(const ProductArgs& a, uint32_t id, uint8_t* ring) {
  if constexpr (TILE == 256) ring_tile_halves<T, TILE, TILE, kAMajor, true>(a, id, ring, StoreEnd<true>());
  else ring_tile<T, TILE, TILE, kAMajor, true>(a, id, ring, StoreEnd<true>());
}

// The gradient's two products in one launch, the one with the longer contraction first (the other's
// workgroups fill the CUs that its last round leaves), and the sum of the row groups' column sums.
template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void gradient_ring(GradientArgs a) {
  __shared__ __align__(1024) uint8_t ring[ring_bytes(TILE)];
  const uint32_t products = a.dx_groups + a.dw_groups;
  uint32_t id = blockIdx.x;
  if (id >= products) return column_sum(a.sums, a.sum_rows, a.n, a.db, id - products, reinterpret_cast<double*>(ring));
  if (a.dw_first) id = id < a.dw_groups ? id + a.dx_groups : id - a.dw_groups;
  if (id < a.dx_groups) gradient_product<T, TILE, false>(a.dx, id, ring);
  else gradient_product<T, TILE, true>(a.dw, id - a.dx_groups, ring);
}

template <typename T, int TILE>
hipError_t layer_for(const ProductArgs& a, hipStream_t s) {
  layer_ring<T, TILE><<<groups_of(a), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int TILE>
hipError_t gradient_for(GradientArgs a, hipStream_t s) {
  a.dx_groups = a.dx.m > 0 ? groups_of(a.dx) : 0;
  a.dw_groups = a.dw.m > 0 ? groups_of(a.dw) : 0;
  const uint32_t columns = a.db ? (uint32_t)((a.n + kSumColumns - 1) / kSumColumns) : 0;
  if (a.dx_groups + a.dw_groups + columns == 0) return hipSuccess;
  gradient_ring<T, TILE><<<a.dx_groups + a.dw_groups + columns, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t layer_type(const ProductArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (a.tile == 256) return layer_for<T, 256>(a, s);
  }
  if (a.tile == 128) return layer_for<T, 128>(a, s);
  return layer_for<T, 64>(a, s);
}

template <typename T>
hipError_t gradient_type(const GradientArgs& a, int tile, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (tile == 256) return gradient_for<T, 256>(a, s);
  }
  if (tile == 128) return gradient_for<T, 128>(a, s);
  return gradient_for<T, 64>(a, s);
}

}  // namespace

hipError_t launch_layer_ring(const ProductArgs& a, hipStream_t s) {
  if (a.type == kBf16) return layer_type<__bf16>(a, s);
  if (a.type == kF16) return layer_type<_Float16>(a, s);
  return layer_type<float>(a, s);
}

hipError_t launch_gradient_ring(const GradientArgs& a, int type, int tile, hipStream_t s) {
  if (type == kBf16) return gradient_type<__bf16>(a, tile, s);
  if (type == kF16) return gradient_type<_Float16>(a, tile, s);
  return gradient_type<float>(a, tile, s);
}

}  // namespace xtvxy
