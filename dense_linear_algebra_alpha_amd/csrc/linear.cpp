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
  bool aligned(int elems) const { return reinterpret_cast<uintptr_t>(p) % (elems * es) == 0 && ld % elems == 0; }
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

// The tile and the number of parts with the least estimated time: a launch and the first loads (3 us),
// the busiest CU's stages, the epilogue (a CU stores a tile at about 8 bytes a cycle; 2 us more for
// 256 x 256, which nothing overlaps), and for parts the sums written and read back at 8 TB/s (they
// stay in the last-level cache) and a second launch.
ProductPlan plan_product(int type, int64_t m, int64_t n, int64_t k, bool ring) {
  ProductPlan best;
  best.k_per_split = std::max<int64_t>(kTileDepth, cdiv(k, kTileDepth) * kTileDepth);
  if (m == 0 || n == 0) return best;
  const int64_t steps = type == kF32 ? 16 : 32;
  double least = 0;
  for (int tile : {64, 128, 256}) {
    if (!ring ? tile != 64 : (tile == 256 && type == kF32)) continue;
    const int64_t tiles = cdiv(m, tile) * cdiv(n, tile);
    for (int64_t splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      const int64_t per = cdiv(cdiv(k, splits), kTileDepth) * kTileDepth;
      if (splits > 1 && (per < 96 || tiles * splits > 16 * kComputeUnits || cdiv(k, per) != splits)) break;
      const int64_t groups = cdiv(tiles * splits, kComputeUnits);
      const double sums = splits > 1 ? 2.0 * splits * m * n * 4 / 8e6 + 2.0 : 0.0;
      const double store = (double)groups * tile * tile * (splits > 1 ? 4 : elem_size(type)) / 8 / 2200 + (tile == 256 ? 2.0 : 0.0);
      const double us = 3.0 + cdiv(per, steps) * stage_us(type, tile, groups) + store + sums;
      if (least == 0 || us < least) {
        least = us;
        best.tile = ring ? tile : 0;
        best.splits = splits;
        best.k_per_split = std::max<int64_t>(per, kTileDepth);
        best.bytes = splits > 1 ? align_up((size_t)splits * m * n * 4) : 0;
      }
    }
  }
  return best;
}

bool product_fits(int64_t m, int64_t n) {
  return cdiv(m, 64) * cdiv(n, 64) <= kMaxGroups && cdiv(m * cdiv(n, 4), 256) <= kMaxGroups;
}

hipError_t run_product(ProductArgs a, const ProductPlan& p, void* ws, hipStream_t s) {
  a.splits = (int32_t)p.splits;
  a.k_per_split = p.k_per_split;
  a.partial = static_cast<float*>(ws);
  hipError_t e = p.tile ? launch_product_ring(a, p.tile, s) : launch_product_tile(a, s);
  if (e == hipSuccess && a.splits > 1) e = launch_product_finish(a, s);
  return e;
}

// A product's operand as the ring kernel takes it: the caller's matrix where its rows are 16-byte
// aligned and whole 16-byte chunks, else a copy in the workspace with rows padded by zeros. Small
// products take any operand as it is.
constexpr int64_t kSmallProduct = (int64_t)1 << 24;  // multiplications

int64_t padded(int64_t cols, int es) { return cdiv(cols, 16 / es) * (16 / es); }

bool whole_chunks(const Matrix& x) {
  return x.aligned16() && x.cols * x.es % 16 == 0 && x.ld * x.es <= kRingMaxPitch;
}

size_t packed_bytes(int64_t rows, int64_t cols, int es) { return align_up((size_t)rows * padded(cols, es) * es); }

bool valid_act(int a) { return a >= XTVXY_ACT_NONE && a <= XTVXY_ACT_SILU; }

// Plan of the layer: whether X and W are copied, the product, and the workspace.
struct LinearPlan {
  bool pack_x = false, pack_w = false;
  ProductPlan product;
  size_t x_off = 0, w_off = 0, partial_off = 0, bytes = 0;
};

LinearPlan plan_linear(int type, int64_t m, int64_t k, int64_t n, bool x_whole, bool w_whole) {
  LinearPlan p;
  const int es = elem_size(type);
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
  a.a_wide = mx.aligned16();
  a.b_wide = mw.aligned16();
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
  const auto wide = [&](int c) { return mo.aligned(c) && (!residual || mr.aligned(c)) && (!pre || mp.aligned(c)); };
  a.e = {bias, residual, ldr, pre, ldp, out, ldo, act, wide(4), wide(8)};
  return status_of(run_product(a, plan.product, base + plan.partial_off, stream));
}

// Plan of the gradient: what is copied, whether d is formed (it is G itself where there is no
// activation and G's rows suit the products), the products, which run one after the other, and the
// workspace: copies of X and W, d, the column sums of the row groups, partial sums.
struct BackwardPlan {
  bool pack_x = false, pack_w = false, form_d = false;
  int64_t ldd = 0, rows_per_group = 0, groups = 0;
  ProductPlan dx, dw;
  size_t x_off = 0, w_off = 0, d_off = 0, sums_off = 0, partial_off = 0, bytes = 0;
};

BackwardPlan plan_backward(int type, int64_t m, int64_t k, int64_t n, int act, bool g_whole, bool x_whole, bool w_whole,
                           bool want_dx, bool want_dw) {
  BackwardPlan p;
  const int es = elem_size(type);
  const bool small = (double)m * n * k < (double)kSmallProduct;
  const bool can = k > 0 && padded(k, es) * es <= kRingMaxPitch && padded(n, 2) * es <= kRingMaxPitch;
  const bool ring_dx = can && (w_whole || !small), ring_dw = can && (x_whole || !small);
  p.pack_w = want_dx && ring_dx && !w_whole;
  p.pack_x = want_dw && ring_dw && !x_whole;
  const bool products = k > 0 && (want_dx || want_dw);
  p.form_d = products && (act != XTVXY_ACT_NONE || (!g_whole && ((want_dx && ring_dx) || (want_dw && ring_dw))));
  p.ldd = cdiv(n, 8) * 8;
  // row groups: about four workgroups per CU, at least 32 rows each
  const int64_t column_groups = std::max<int64_t>(1, cdiv(n, 512));
  const int64_t groups = std::max<int64_t>(1, 4 * kComputeUnits / column_groups);
  p.rows_per_group = std::max<int64_t>(32, cdiv(m, groups));
  p.groups = std::max<int64_t>(1, cdiv(m, p.rows_per_group));
  p.dx = plan_product(type, m, k, n, ring_dx);
  p.dw = plan_product(type, n, k, m, ring_dw);
  const auto take = [&](bool want, size_t bytes) {
    const size_t at = p.bytes;
    if (want) p.bytes += bytes;
    return at;
  };
  p.x_off = take(p.pack_x, packed_bytes(m, k, es));
  p.w_off = take(p.pack_w, packed_bytes(n, k, es));
  p.d_off = take(p.form_d, align_up((size_t)m * p.ldd * es));
  p.sums_off = take(true, align_up((size_t)p.groups * n * 4));
  p.partial_off = take(products, std::max(want_dx ? p.dx.bytes : 0, want_dw ? p.dw.bytes : 0));
  return p;
}

bool backward_fits(int64_t m, int64_t k, int64_t n) {
  return product_fits(m, k) && product_fits(n, k) && cdiv(n, 512) <= kMaxGroups / 2048;
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
  hipError_t e = hipSuccess;
  const void* D = G;
  int64_t ldd = ldg;
  if (reads && (p.form_d || db)) {
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
    s.wide = mg.aligned16() && (!pre || mp.aligned16());
    s.sums = db ? reinterpret_cast<float*>(base + p.sums_off) : nullptr;
    s.rows_per_group = p.rows_per_group;
    s.groups = p.groups;
    e = launch_slope(s, stream);
    if (e == hipSuccess && db) e = launch_column_finish(s.sums, s.groups, n, db, stream);
  } else if (db && n > 0) {
    e = launch_zero(db, (size_t)n * 4, stream);
  }
  if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  if (p.form_d) {
    D = base + p.d_off;
    ldd = p.ldd;
  }
  PackArgs pack{};
  if (reads && p.pack_x) pack.job[pack.jobs++] = {X, base + p.x_off, ldx, padded(k, es), m, k};
  if (reads && p.pack_w) pack.job[pack.jobs++] = {W, base + p.w_off, ldw, padded(k, es), n, k};
  if (pack.jobs > 0 && launch_pack(pack, type, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  const Matrix md{D, m, n, ldd, es};
  ProductArgs a{};
  a.A = D;
  a.lda = ldd;
  a.a_wide = md.aligned16();
  a.b_contraction_major = 1;
  a.n = k;
  a.type = type;
  if (dX && m > 0 && k > 0) {
    a.B = p.pack_w && reads ? base + p.w_off : W;
    a.ldb = p.pack_w ? padded(k, es) : ldw;
    a.b_wide = p.pack_w || mw.aligned16();
    a.m = m;
    a.k = n;
    a.e = {nullptr, nullptr, 0, nullptr, 0, dX, lddx, XTVXY_ACT_NONE, mdx.aligned(4), mdx.aligned(8)};
    e = run_product(a, p.dx, base + p.partial_off, stream);
    if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  if (dW && n > 0 && k > 0) {
    a.a_contraction_major = 1;
    a.B = p.pack_x && reads ? base + p.x_off : X;
    a.ldb = p.pack_x ? padded(k, es) : ldx;
    a.b_wide = p.pack_x || mx.aligned16();
    a.m = n;
    a.k = m;
    a.e = {nullptr, nullptr, 0, nullptr, 0, dW, lddw, XTVXY_ACT_NONE, mdw.aligned(4), mdw.aligned(8)};
    e = run_product(a, p.dw, base + p.partial_off, stream);
    if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  return XTVXY_SUCCESS;
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
