// Internal declarations of the fully connected layer (linear.cpp, linear_*.hip): the products
// X W^T, D W and D^T X with what follows them, and the gradient through the activation.
#pragma once

#include "internal.h"

namespace xtvxy {

enum ElemType { kF32 = 0, kBf16 = 1, kF16 = 2 };
constexpr int elem_size(int t) { return t == kF32 ? 4 : 2; }

// What is done with a product's sums z[i][j] (fp32) before they are stored:
//   z += bias[j]; pre[i][j] = z; out[i][j] = act(z) + residual[i][j].
// bias, pre and residual may be null; residual, pre and out have the product's element type.
struct LinearEpilogue {
  const float* bias;
  const void* residual;
  int64_t ldr;
  void* pre;
  int64_t ldp;
  void* out;
  int64_t ldo;
  int32_t act;     // XTVXY_ACT_*
};

// C[i][j] = sum over k of A(i, k) B(j, k), i < m, j < n, followed by the epilogue. Where
// a_contraction_major, A(i, k) = A[k * lda + i], else A[i * lda + k]; B likewise.
struct ProductArgs {
  const void* A;
  const void* B;
  int64_t lda, ldb;
  int64_t m, n, k;
  int32_t type;
  int32_t a_contraction_major, b_contraction_major;
  int32_t tile;             // edge of the ring kernel's tiles, 0 for the other kernels
  // The first `whole` tiles (in the order of tile_of) run over the whole contraction; the others are
  // split into parts of it, each with sums of its own in `partial`: [splits][other tiles][tile][tile].
  // The other kernels split everything (whole 0): [splits][m][n].
  int32_t splits;
  int64_t whole;
  int64_t k_per_split;      // a multiple of the tile's depth; splits * k_per_split >= k
  float* partial;           // used when splits > 1 or in_parts
  int32_t in_parts;         // nonzero: sums in one part go to `partial` too (ring kernel with whole 0, few rows)
  const float* scale;       // on the device: of the sums of a gradient's product, null for 1
  __host__ __device__ int64_t tiles() const { return ((m + tile - 1) / tile) * ((n + tile - 1) / tile); }
  LinearEpilogue e;
};

constexpr int kTileDepth = 32;   // contraction steps of the 64 x 64 tile kernel
// The layer's product (both contractions contiguous) at any size and alignment.
hipError_t launch_layer_tile(const ProductArgs& a, hipStream_t s);

// Operands with 16-byte aligned rows of at most kRingMaxPitch bytes; what lies between a row's end and
// the next multiple of 16 bytes is zero where the contraction is contiguous, and readable where it is
// not. a.tile: 64, 128, or 256 (16-bit elements). k_per_split is a multiple of 32.
constexpr int64_t kRingMaxPitch = (int64_t)1 << 22;  // 256 rows stay within 32-bit offsets
hipError_t launch_layer_ring(const ProductArgs& a, hipStream_t s);

// The gradient's products dX = d W (d contraction-contiguous, W strided) and dW = d^T X (both
// strided), either with m == 0 where it is not wanted, and db[j] = the sum over sum_rows of
// sums[.][n] (db null: not wanted).
struct GradientArgs {
  ProductArgs dx, dw;
  uint32_t dx_groups, dw_groups;  // workgroups (set by the launcher)
  int32_t dw_first;               // the ring kernel starts dw's workgroups first
  const float* sums;
  int64_t sum_rows, n;
  float* db;
  // the tile kernel forms d itself: dx.A and dw.A are G, and
  const void* pre;    // null: slope 1
  int64_t ldp;
  int32_t act;
  float* own_sums;    // [dw.splits][n] column sums of d, or null
};
hipError_t launch_gradient_ring(const GradientArgs& a, int type, int tile, hipStream_t s);
// At any size and alignment, d formed as it is loaded. (db is left to launch_gradient_finish.)
hipError_t launch_gradient_tile(const GradientArgs& a, int type, hipStream_t s);
// Sums the parts of split products, and the column sums' rows, each in ascending order.
hipError_t launch_gradient_finish(const GradientArgs& a, int type, hipStream_t s);

// At most kFewRows rows of A, both operands with the contraction contiguous, at any alignment. A
// workgroup of `waves` (4 or 8) wavefronts takes `outputs` (16 or 32) rows of B; each wavefront of
// each split takes k_per_split steps, a multiple of 32: splits * waves * k_per_split >= k.
constexpr int64_t kFewRows = 32;
hipError_t launch_product_few(const ProductArgs& a, int waves, int outputs, hipStream_t s);
// Copies of up to kPackJobs matrices with rows of ldd elements (a multiple of 16 bytes, at least
// cols), zero beyond cols.
constexpr int kPackJobs = 4;
struct PackJob {
  const void* src;
  void* dst;
  int64_t ld, ldd, rows, cols;
};
struct PackArgs {
  PackJob job[kPackJobs];
  int32_t jobs;
};
hipError_t launch_pack(const PackArgs& a, int type, hipStream_t s);
// Sums the parts of a split product in ascending order and applies the epilogue.
hipError_t launch_product_finish(const ProductArgs& a, hipStream_t s);

// d = g * act'(pre) (d may be null: column sums only; pre null: slope 1), and per-workgroup
// column sums of the unrounded d: sums[groups][n]. Rows of d are zero from n up to ldd.
struct SlopeArgs {
  const void* g;
  const void* pre;
  void* d;
  int64_t ldg, ldp, ldd;
  int64_t m, n;
  int32_t type, act;
  float* sums;           // null: no column sums
  int64_t rows_per_group, groups;
};
constexpr int64_t kSlopeNarrow = 256;  // columns up to which a workgroup takes 128 instead of 512
hipError_t launch_slope(const SlopeArgs& a, hipStream_t s);

}  // namespace xtvxy
