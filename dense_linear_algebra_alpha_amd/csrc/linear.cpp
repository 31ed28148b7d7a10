// Host side of the fully connected layer and its gradient: argument checks, the choice of kernels
// and the workspace, and the launches. Argument errors are found before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "linear.h"

using namespace xtvxy;

namespace {

constexpr int64_t kComputeUnits = 256;           // the plans are for this chip whatever runs the query
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads in one launch: below 2^32 threads

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool bytes_overflow(int64_t rows, int64_t ld) { return rows > 0 && ld > INT64_MAX / 16 / rows; }

struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
  int es;
  size_t extent() const { return rows > 0 && cols > 0 ? (size_t)((rows - 1) * ld + cols) * es : 0; }
  bool aligned16() const { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0; }
};

// Whether two matrices share an element (rows of equal pitch: exact; else by their extents).
bool overlap(const Matrix& a, const Matrix& b) {
  if (!a.p || !b.p) return false;
  const size_t an = a.extent(), bn = b.extent();
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (an == 0 || bn == 0 || x >= y + bn || y >= x + an) return false;
  const int64_t pitch = a.ld * a.es;
  if (pitch != b.ld * b.es) return true;
  int64_t d = (int64_t)(y - x) % pitch;  // of b's first column past a's, around the pitch
  if (d < 0) d += pitch;
  return !(d >= a.cols * a.es && d + b.cols * b.es <= pitch);
}

Matrix vec(const float* p, int64_t n) { return {p, 1, n, n > 0 ? n : 1, 4}; }

xtvxy_status status_of(hipError_t e) { return e == hipSuccess ? XTVXY_SUCCESS : XTVXY_ERROR_LAUNCH; }

// How one product is computed: by which kernel, and in how many parts of the contraction.
struct ProductPlan {
  int tile = 0;  // 0: the kernel for any alignment; 64, 128, 256: the ring kernel's tile
  int64_t splits = 1, k_per_split = 0;
  size_t bytes = 0;  // partial sums
};

// Microseconds per stage of a CU that runs `groups` workgroups of a tile in all, of which several are
// resident at once (one of 256, two of 128, five of 64). Measured on products of 2^28 .. 2^40
// multiplications: 256 x 256 0.88 (the matrix unit is busy), 128 x 128 0.33 for a lone workgroup and
// 0.57 for two, 64 x 64 0.18 alone and 0.13 each from two on; fp32 stages take the matrix unit 3.4, 0.84
// (128, 64; half the contraction steps of a 16-bit stage).
double stage_us(int type, int tile, int64_t groups) {
  if (type == kF32) return tile == 128 ? 1.18 * groups : (groups <= 1 ? 0.36 : 0.28 * groups);
  if (tile == 256) return 0.88 * groups;
  if (tile == 128) return groups <= 1 ? 0.33 : 0.285 * groups;
  return groups <= 1 ? 0.18 : 0.13 * groups;
}

// Times and sizes of one product with a tile and a number of parts. Estimated: the stages (launch and
// first loads are not counted), the epilogue's stores (a CU stores a tile at about 8 bytes a cycle),
// and for parts the sums written and read back at 8 TB/s (they stay in the last-level cache).
struct ProductCost {
  int64_t groups = 0, stages = 0, per = 0;
  double extra_us = 0;
};
bool product_cost(int type, int tile, int64_t splits, int64_t m, int64_t n, int64_t k, ProductCost* c) {
  *c = {};
  c->per = std::max<int64_t>(kTileDepth, cdiv(cdiv(k, splits), kTileDepth) * kTileDepth);
  const int64_t tiles = cdiv(m, tile) * cdiv(n, tile);
  if (splits > 1 && (c->per < 64 || tiles * splits > 16 * kComputeUnits || cdiv(k, c->per) != splits)) return false;
  c->groups = tiles * splits;
  c->stages = cdiv(c->per, type == kF32 ? 16 : 32);
  c->extra_us = (double)cdiv(c->groups, kComputeUnits) * tile * tile * (splits > 1 ? 4 : elem_size(type)) / 8 / 2200 +
                (tile == 256 ? 2.0 : 0.0) + (splits > 1 ? 2.0 * splits * m * n * 4 / 8e6 : 0.0);
  return true;
}

constexpr int64_t kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

void set_product(ProductPlan* p, int tile, int64_t splits, const ProductCost& c, int64_t m, int64_t n) {
  p->tile = tile;
  p->splits = splits;
  p->k_per_split = c.per;
  p->bytes = splits > 1 ? align_up((size_t)splits * m * n * 4) : 0;
}

// The layer's tile and number of parts with the least estimated time (2 us for the second launch of a
// split product).
ProductPlan plan_product(int type, int64_t m, int64_t n, int64_t k, bool ring) {
  ProductPlan best;
  best.k_per_split = kTileDepth;
  if (m == 0 || n == 0) return best;
  double least = 0;
  for (int tile : {64, 128, 256}) {
    if (!ring ? tile != 64 : (tile == 256 && type == kF32)) continue;
    for (int64_t splits : kSplits) {
      ProductCost c;
      if (!product_cost(type, tile, splits, m, n, k, &c)) continue;
      const double us = c.stages * stage_us(type, tile, cdiv(c.groups, kComputeUnits)) + c.extra_us + (splits > 1 ? 2.0 : 0.0);
      if (least == 0 || us < least) {
        least = us;
        set_product(&best, ring ? tile : 0, splits, c, m, n);
      }
    }
  }
  return best;
}

// The gradient's products dX (m x k, contraction n) and dW (n x k, contraction m) share a tile and a
// launch: the CUs' stages are those of both, and at least the longer product's.
void plan_gradient(int type, int64_t m, int64_t k, int64_t n, bool want_dx, bool want_dw, bool ring, ProductPlan* dx,
                   ProductPlan* dw) {
  dx->k_per_split = dw->k_per_split = kTileDepth;
  if (m == 0 || k == 0 || n == 0) return;
  double least = 0;
  for (int tile : {64, 128, 256}) {
    if (!ring ? tile != 64 : (tile == 256 && type == kF32)) continue;
    for (int64_t sx : kSplits) {
      ProductCost cx, cw;
      if (want_dx ? !product_cost(type, tile, sx, m, k, n, &cx) : sx > 1) continue;
      for (int64_t sw : kSplits) {
        if (want_dw ? !product_cost(type, tile, sw, n, k, m, &cw) : sw > 1) continue;
        const int64_t groups = cx.groups + cw.groups, rounds = cdiv(groups, kComputeUnits);
        const double mean = (double)(cx.groups * cx.stages + cw.groups * cw.stages) / groups;
        const double longest = (double)std::max(cx.stages, cw.stages) * stage_us(type, tile, 1);
        const double us = std::max(longest, mean * stage_us(type, tile, rounds)) + cx.extra_us + cw.extra_us +
                          (sx > 1 || sw > 1 ? 2.0 : 0.0);
        if (least == 0 || us < least) {
          least = us;
          if (want_dx) set_product(dx, ring ? tile : 0, sx, cx, m, k);
          if (want_dw) set_product(dw, ring ? tile : 0, sw, cw, n, k);
        }
      }
    }
  }
}

bool product_fits(int64_t m, int64_t n) {
  return cdiv(m, 64) * cdiv(n, 64) <= kMaxGroups;
}

hipError_t run_layer(ProductArgs a, const ProductPlan& p, void* ws, hipStream_t s) {
  a.splits = (int32_t)p.splits;
  a.k_per_split = p.k_per_split;
  a.partial = static_cast<float*>(ws);
  hipError_t e = p.tile ? launch_layer_ring(a, p.tile, s) : launch_layer_tile(a, s);
  if (e == hipSuccess && a.splits > 1) e = launch_product_finish(a, s);
  return e;
}

// A product's operand as the ring kernel takes it: the caller's matrix where its rows are 16-byte
// aligned and whole 16-byte chunks, else a copy in the workspace with rows padded by zeros. Small
// products take any operand as it is.
constexpr int64_t kSmallProduct = (int64_t)1 << 24;  // multiplications
constexpr int64_t kSmallGradient = (int64_t)1 << 26;

int64_t padded(int64_t cols, int es) { return cdiv(cols, 16 / es) * (16 / es); }

bool whole_chunks(const Matrix& x) {
  return x.aligned16() && x.cols * x.es % 16 == 0 && x.ld * x.es <= kRingMaxPitch;
}

size_t packed_bytes(int64_t rows, int64_t cols, int es) { return align_up((size_t)rows * padded(cols, es) * es); }

bool valid_act(int a) { return a >= XTVXY_ACT_NONE && a <= XTVXY_ACT_SILU; }

// Plan of the layer: whether X and W are copied, the product, and the workspace.
struct LinearPlan {
  bool pack_x = false, pack_w = false;
  int few = 0, few_outputs = 0;  // the kernel for few rows: its wavefronts, its outputs of a workgroup
  ProductPlan product;
  size_t x_off = 0, w_off = 0, partial_off = 0, bytes = 0;
};

LinearPlan plan_linear(int type, int64_t m, int64_t k, int64_t n, bool x_whole, bool w_whole) {
  LinearPlan p;
  const int es = elem_size(type);
  if (m <= kFewRows) {
    // W cold, us: 16 outputs a workgroup against 32: 1 x 4096 x 4096 bf16 8.9, 11.9; 13 x 2048 x 8192 11.2, 10.5
    // (X is loaded once per workgroup); 4 wavefronts against 8: bf16 8.9, 9.5, fp32 18.1, 16.9. Where the
    // outputs are too few for the CUs the contraction is split: 1 x 8192 x 1024 12.1 to 9.7, 1 x 16384 x 256
    // 20.1 to 9.0. The ring kernel with its best split: 13.9, 14.8, 13.9, 27.4, 13.2, 15.4; at 32 rows of
    // 4096 x 4096 15.6 against 14.7, at 48 14.9 against 21.
    p.few_outputs = m > 4 && n >= 8192 ? 32 : 16;
    const int64_t groups = cdiv(n, p.few_outputs);
    p.few = k >= 4096 && (type == kF32 || groups < kComputeUnits) ? 8 : 4;
    int64_t splits = 1;
    if (groups <= kComputeUnits / 2 && k * es >= 16384)
      splits = std::max<int64_t>(1, std::min<int64_t>({8, kComputeUnits / groups, k / (p.few * 256)}));
    p.product.k_per_split = std::max<int64_t>(32, cdiv(cdiv(k, p.few * splits), 32) * 32);
    p.product.splits = std::max<int64_t>(1, cdiv(k, p.few * p.product.k_per_split));
    if (p.product.splits > 1) p.bytes = p.product.bytes = align_up((size_t)p.product.splits * m * n * 4);
    return p;
  }
  const bool small = (double)m * n * k < (double)kSmallProduct;
  const bool ring = (x_whole && w_whole) || (!small && k > 0 && padded(k, es) * es <= kRingMaxPitch);
  p.pack_x = ring && !x_whole;
  p.pack_w = ring && !w_whole;
  p.product = plan_product(type, m, n, k, ring);
  if (p.pack_x) {
    p.x_off = p.bytes;
    p.bytes += packed_bytes(m, k, es);
  }
  if (p.pack_w) {
    p.w_off = p.bytes;
    p.bytes += packed_bytes(n, k, es);
  }
  p.partial_off = p.bytes;
  p.bytes += p.product.bytes;
  return p;
}

xtvxy_status linear_workspace(int type, int64_t m, int64_t k, int64_t n, int aligned16, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || k < 0 || n < 0) return XTVXY_ERROR_INVALID_VALUE;
  if (bytes_overflow(m, n) || bytes_overflow(m, k + 8) || bytes_overflow(n, k + 8)) return XTVXY_ERROR_INVALID_VALUE;
  *bytes = 0;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!product_fits(m, n)) return XTVXY_ERROR_UNSUPPORTED;
  // of X and W either may turn out to need its copy where aligned16 is 0: the largest of the plans
  const bool chunks = k * elem_size(type) % 16 == 0;
  for (int x = 0; x < 2; ++x)
    for (int w = 0; w < 2; ++w)
      if (!aligned16 || !chunks || (x && w))
        *bytes = std::max(*bytes, plan_linear(type, m, k, n, chunks && x, chunks && w).bytes);
  return XTVXY_SUCCESS;
}

bool bad_ld(int64_t ld, int64_t cols, int64_t rows) { return ld < std::max<int64_t>(cols, 1) || bytes_overflow(rows, ld); }

xtvxy_status linear_impl(int type, int64_t m, int64_t k, int64_t n, const void* X, int64_t ldx, const void* W,
                         int64_t ldw, const float* bias, const void* residual, int64_t ldr, int act, void* out,
                         int64_t ldo, void* pre, int64_t ldp, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (m < 0 || k < 0 || n < 0 || !valid_act(act)) return XTVXY_ERROR_INVALID_VALUE;
  if (bad_ld(ldx, k, m) || bad_ld(ldw, k, n) || bad_ld(ldo, n, m) || (residual && bad_ld(ldr, n, m)) ||
      (pre && bad_ld(ldp, n, m)))
    return XTVXY_ERROR_INVALID_VALUE;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!out || (k > 0 && (!X || !W))) return XTVXY_ERROR_NULL_POINTER;
  if (!product_fits(m, n)) return XTVXY_ERROR_UNSUPPORTED;
  const int es = elem_size(type);
  const Matrix mx{X, m, k, ldx, es}, mw{W, n, k, ldw, es}, mr{residual, m, n, ldr, es}, mo{out, m, n, ldo, es},
      mp{pre, m, n, ldp, es}, mb = vec(bias, n);
  if (overlap(mo, mx) || overlap(mo, mw) || overlap(mo, mb) || overlap(mo, mp) || overlap(mp, mx) || overlap(mp, mw) ||
      overlap(mp, mb) || overlap(mp, mr))
    return XTVXY_ERROR_ALIASING;
  if (residual && !(residual == out && ldr == ldo) && overlap(mo, mr)) return XTVXY_ERROR_ALIASING;
  const LinearPlan plan = plan_linear(type, m, k, n, whole_chunks(mx), whole_chunks(mw));
  if (plan.bytes > 0 && (!ws || ws_bytes < plan.bytes || reinterpret_cast<uintptr_t>(ws) % kAlign != 0))
    return XTVXY_ERROR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  ProductArgs a{};
  a.A = X;
  a.B = W;
  a.lda = ldx;
  a.ldb = ldw;
  a.m = m;
  a.n = n;
  a.k = k;
  a.type = type;
  PackArgs pack{};
  if (plan.pack_x) {
    pack.job[pack.jobs++] = {X, base + plan.x_off, ldx, padded(k, es), m, k};
    a.A = base + plan.x_off;
    a.lda = padded(k, es);
  }
  if (plan.pack_w) {
    pack.job[pack.jobs++] = {W, base + plan.w_off, ldw, padded(k, es), n, k};
    a.B = base + plan.w_off;
    a.ldb = padded(k, es);
  }
  if (pack.jobs > 0 && launch_pack(pack, type, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  a.e = {bias, residual, ldr, pre, ldp, out, ldo, act};
  if (plan.few) {
    a.splits = (int32_t)plan.product.splits;
    a.k_per_split = plan.product.k_per_split;
    a.partial = reinterpret_cast<float*>(base);
    hipError_t e = launch_product_few(a, plan.few, plan.few_outputs, stream);
    if (e == hipSuccess && a.splits > 1) e = launch_product_finish(a, stream);
    return status_of(e);
  }
  return status_of(run_layer(a, plan.product, base + plan.partial_off, stream));
}

// Plan of the gradient. Small ones form d as they load G and pre (`fused`: one launch, and one for
// parts and column sums). Others first form d in the workspace (it is G itself where there is no
// activation and G's rows suit the products) with the column sums of row groups, copy X and W where
// their rows do not suit, and then run both products in one launch. Workspace: copies of X and W, d,
// column sums, partial sums of dX and of dW.
struct BackwardPlan {
  bool fused = false, pack_x = false, pack_w = false, form_d = false;
  int64_t ldd = 0, rows_per_group = 0, groups = 0;
  ProductPlan dx, dw;
  size_t x_off = 0, w_off = 0, d_off = 0, sums_off = 0, dx_off = 0, dw_off = 0, bytes = 0;
};

BackwardPlan plan_backward(int type, int64_t m, int64_t k, int64_t n, int act, bool g_whole, bool x_whole, bool w_whole,
                           bool want_dx, bool want_dw) {
  BackwardPlan p;
  const int es = elem_size(type);
  want_dx = want_dx && k > 0;
  want_dw = want_dw && k > 0;
  const bool fits_ring = padded(k, es) * es <= kRingMaxPitch && cdiv(n, 8) * 8 * es <= kRingMaxPitch;
  // us on fp32, fused against not: 2048 x 128 x 64 17.3, 16.0 (and a launch less), 512 x 256 x 256 11.4, 14.5,
  // 1024 x 256 x 256 13.4, 16.5, 1024 x 512 x 256 17.5, 18.5, 1501 x 1000 x 501 54, 49; 16-bit loses at
  // every size (the tile kernel turns strided operands element by element): 512 x 256 x 256 20.5, 10.2
  p.fused = (want_dx || want_dw) && (!fits_ring || (type == kF32 && (double)m * n * k <= (double)kSmallGradient));
  const bool ring = (want_dx || want_dw) && !p.fused;
  p.pack_w = want_dx && ring && !w_whole;
  p.pack_x = want_dw && ring && !x_whole;
  p.form_d = ring && (act != XTVXY_ACT_NONE || !g_whole);
  p.ldd = cdiv(n, 8) * 8;
  // row groups: about four workgroups per CU, at least 2 rows for each row that a workgroup takes at once
  const bool narrow = n <= kSlopeNarrow;
  const int64_t column_groups = std::max<int64_t>(1, cdiv(n, narrow ? 128 : 512));
  const int64_t groups = std::max<int64_t>(1, 4 * kComputeUnits / column_groups);
  p.rows_per_group = std::max<int64_t>(narrow ? 32 : 8, cdiv(m, groups));
  p.groups = std::max<int64_t>(1, cdiv(m, p.rows_per_group));
  plan_gradient(type, m, k, n, want_dx, want_dw, ring, &p.dx, &p.dw);
  const auto take = [&](bool want, size_t bytes) {
    const size_t at = p.bytes;
    if (want) p.bytes += bytes;
    return at;
  };
  p.x_off = take(p.pack_x, packed_bytes(m, k, es));
  p.w_off = take(p.pack_w, packed_bytes(n, k, es));
  p.d_off = take(p.form_d, align_up((size_t)m * p.ldd * es));
  p.sums_off = take(true, align_up((size_t)std::max(p.groups, p.fused ? p.dw.splits : 0) * n * 4));
  p.dx_off = take(want_dx, p.dx.bytes);
  p.dw_off = take(want_dw, p.dw.bytes);
  return p;
}

bool backward_fits(int64_t m, int64_t k, int64_t n) {
  // both products are one launch
  return cdiv(m, 64) * cdiv(k, 64) + cdiv(n, 64) * cdiv(k, 64) + cdiv(n, 16) <= kMaxGroups;
}

xtvxy_status backward_workspace(int type, int64_t m, int64_t k, int64_t n, int act, int aligned16, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || k < 0 || n < 0 || !valid_act(act)) return XTVXY_ERROR_INVALID_VALUE;
  if (bytes_overflow(m, n + 8) || bytes_overflow(m, k + 8) || bytes_overflow(n, k + 8)) return XTVXY_ERROR_INVALID_VALUE;
  *bytes = 0;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!backward_fits(m, k, n)) return XTVXY_ERROR_UNSUPPORTED;
  // any of G, X and W may turn out to need its copy where aligned16 is 0: the largest of the plans
  const int es = elem_size(type);
  const bool kc = k * es % 16 == 0, nc = n * es % 16 == 0;
  for (int c = 0; c < 8; ++c) {
    const bool g = c & 1, x = c & 2, w = c & 4;
    if (aligned16 && !(g == nc && x == kc && w == kc)) continue;
    *bytes = std::max(*bytes, plan_backward(type, m, k, n, act, nc && g, kc && x, kc && w, true, true).bytes);
  }
  return XTVXY_SUCCESS;
}

xtvxy_status backward_impl(int type, int64_t m, int64_t k, int64_t n, const void* G, int64_t ldg, const void* X,
                           int64_t ldx, const void* W, int64_t ldw, const void* pre, int64_t ldp, int act, void* dX,
                           int64_t lddx, void* dW, int64_t lddw, float* db, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  if (m < 0 || k < 0 || n < 0 || !valid_act(act)) return XTVXY_ERROR_INVALID_VALUE;
  if (bytes_overflow(m, n + 8)) return XTVXY_ERROR_INVALID_VALUE;
  if (bad_ld(ldg, n, m) || bad_ld(ldx, k, m) || bad_ld(ldw, k, n) || (dX && bad_ld(lddx, k, m)) ||
      (dW && bad_ld(lddw, k, n)) || (act != XTVXY_ACT_NONE && bad_ld(ldp, n, m)))
    return XTVXY_ERROR_INVALID_VALUE;
  const bool reads = m > 0 && n > 0 && (dX || dW || db);
  if (reads && (!G || (act != XTVXY_ACT_NONE && !pre) || (dX && k > 0 && !W) || (dW && k > 0 && !X)))
    return XTVXY_ERROR_NULL_POINTER;
  if (!backward_fits(m, k, n)) return XTVXY_ERROR_UNSUPPORTED;
  if (act == XTVXY_ACT_NONE) pre = nullptr;
  const int es = elem_size(type);
  const Matrix mg{G, m, n, ldg, es}, mx{X, m, k, ldx, es}, mw{W, n, k, ldw, es}, mp{pre, m, n, ldp, es},
      mdx{dX, m, k, lddx, es}, mdw{dW, n, k, lddw, es}, mdb = vec(db, n);
  for (const Matrix* o : {&mdx, &mdw, &mdb})
    for (const Matrix* i : {&mg, &mx, &mw, &mp})
      if (overlap(*o, *i)) return XTVXY_ERROR_ALIASING;
  if (overlap(mdx, mdw) || overlap(mdx, mdb) || overlap(mdw, mdb)) return XTVXY_ERROR_ALIASING;

  const BackwardPlan p = plan_backward(type, m, k, n, act, whole_chunks(mg), whole_chunks(mx), whole_chunks(mw),
                                       dX != nullptr, dW != nullptr);
  if (reads && p.bytes > 0 && (!ws || ws_bytes < p.bytes || reinterpret_cast<uintptr_t>(ws) % kAlign != 0))
    return XTVXY_ERROR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  GradientArgs a{};
  a.n = n;
  a.db = db;
  a.sums = reinterpret_cast<const float*>(base + p.sums_off);
  if (dX && k > 0) {
    a.dx.B = W;
    a.dx.ldb = ldw;
    a.dx.m = m;
    a.dx.n = k;
    a.dx.k = n;
    a.dx.splits = (int32_t)p.dx.splits;
    a.dx.k_per_split = p.dx.k_per_split;
    a.dx.partial = reinterpret_cast<float*>(base + p.dx_off);
    a.dx.e = {nullptr, nullptr, 0, nullptr, 0, dX, lddx, XTVXY_ACT_NONE};
  }
  if (dW && k > 0) {
    a.dw.B = X;
    a.dw.ldb = ldx;
    a.dw.m = n;
    a.dw.n = k;
    a.dw.k = m;
    a.dw.splits = (int32_t)p.dw.splits;
    a.dw.k_per_split = p.dw.k_per_split;
    a.dw.partial = reinterpret_cast<float*>(base + p.dw_off);
    a.dw.e = {nullptr, nullptr, 0, nullptr, 0, dW, lddw, XTVXY_ACT_NONE};
  }
  a.dx.type = a.dw.type = type;
  a.dx.A = a.dw.A = G;
  a.dx.lda = a.dw.lda = ldg;
  if (!reads) {  // no rows or no outputs: db is zero, and so are the products' empty sums
    if (db && n > 0 && launch_zero(db, (size_t)n * 4, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    return status_of(launch_gradient_tile(a, type, stream));
  }
  if (p.fused && (dW || !db)) {
    a.pre = pre;
    a.ldp = ldp;
    a.act = act;
    a.own_sums = db ? reinterpret_cast<float*>(base + p.sums_off) : nullptr;
    a.sum_rows = p.dw.splits;
    if (launch_gradient_tile(a, type, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    return status_of(launch_gradient_finish(a, type, stream));
  }
  if (p.form_d || db) {
    SlopeArgs s{};
    s.g = G;
    s.ldg = ldg;
    s.pre = pre;
    s.ldp = ldp;
    s.d = p.form_d ? base + p.d_off : nullptr;
    s.ldd = p.ldd;
    s.m = m;
    s.n = n;
    s.type = type;
    s.act = act;
    s.sums = db ? reinterpret_cast<float*>(base + p.sums_off) : nullptr;
    s.rows_per_group = p.rows_per_group;
    s.groups = p.groups;
    if (launch_slope(s, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    a.sum_rows = p.groups;
  }
  if (p.fused) {  // db without dW: the column sums are the row groups'
    a.pre = pre;
    a.ldp = ldp;
    a.act = act;
    if (launch_gradient_tile(a, type, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    return status_of(launch_gradient_finish(a, type, stream));
  }
  if (p.form_d) {
    a.dx.A = a.dw.A = base + p.d_off;
    a.dx.lda = a.dw.lda = p.ldd;
  }
  PackArgs pack{};
  if (p.pack_x) {
    pack.job[pack.jobs++] = {X, base + p.x_off, ldx, padded(k, es), m, k};
    a.dw.B = base + p.x_off;
    a.dw.ldb = padded(k, es);
  }
  if (p.pack_w) {
    pack.job[pack.jobs++] = {W, base + p.w_off, ldw, padded(k, es), n, k};
    a.dx.B = base + p.w_off;
    a.dx.ldb = padded(k, es);
  }
  if (pack.jobs > 0 && launch_pack(pack, type, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  // the products and db in one launch; with parts the sums are finished in a second one
  if (launch_gradient_ring(a, type, dX && k > 0 ? p.dx.tile : p.dw.tile, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  a.db = nullptr;
  return status_of(launch_gradient_finish(a, type, stream));
}

}  // namespace

extern "C" {

#define XTVXY_LINEAR(SUFFIX, TYPE, T)                                                                                 \
  xtvxy_status xtvxy_linear_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n, int aligned16, size_t* bytes) { \
    return linear_workspace(TYPE, m, k, n, aligned16, bytes);                                                         \
  }                                                                                                                   \
  xtvxy_status xtvxy_linear_##SUFFIX(int64_t m, int64_t k, int64_t n, const T* X, int64_t ldx, const T* W,            \
                                     int64_t ldw, const float* bias, const T* residual, int64_t ldr, int activation,  \
                                     T* out, int64_t ldo, T* pre, int64_t ldp, void* workspace,                       \
                                     size_t workspace_bytes, hipStream_t stream) {                                    \
    return linear_impl(TYPE, m, k, n, X, ldx, W, ldw, bias, residual, ldr, activation, out, ldo, pre, ldp, workspace, \
                       workspace_bytes, stream);                                                                      \
  }                                                                                                                   \
  xtvxy_status xtvxy_linear_backward_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n, int activation,       \
                                                               int aligned16, size_t* bytes) {                        \
    return backward_workspace(TYPE, m, k, n, activation, aligned16, bytes);                                           \
  }                                                                                                                   \
  xtvxy_status xtvxy_linear_backward_##SUFFIX(int64_t m, int64_t k, int64_t n, const T* G, int64_t ldg, const T* X,   \
                                              int64_t ldx, const T* W, int64_t ldw, const T* pre, int64_t ldp,        \
                                              int activation, T* dX, int64_t lddx, T* dW, int64_t lddw, float* db,    \
                                              void* workspace, size_t workspace_bytes, hipStream_t stream) {          \
    return backward_impl(TYPE, m, k, n, G, ldg, X, ldx, W, ldw, pre, ldp, activation, dX, lddx, dW, lddw, db,         \
                         workspace, workspace_bytes, stream);                                                         \
  }

XTVXY_LINEAR(f32, kF32, float)
XTVXY_LINEAR(bf16, kBf16, uint16_t)
XTVXY_LINEAR(f16, kF16, uint16_t)

}  // extern "C"
