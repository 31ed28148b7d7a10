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
  bool aligned4() const { return reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && ld % 4 == 0; }
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

// How one product is computed: workspace and split of the contraction.
struct ProductPlan {
  int64_t splits = 1, k_per_split = 0;
  size_t bytes = 0;  // partial sums
};

// Splits of the contraction: enough workgroups for two per CU, each part at least 8 tile depths.
ProductPlan plan_product(int64_t m, int64_t n, int64_t k) {
  ProductPlan p;
  p.k_per_split = k > 0 ? k : kTileDepth;
  const int64_t tiles = cdiv(m, 64) * cdiv(n, 64);
  int64_t want = tiles > 0 ? 2 * kComputeUnits / tiles : 1;
  want = std::min(want, k / (8 * kTileDepth));
  if (want > 1) {
    p.k_per_split = cdiv(cdiv(k, want), kTileDepth) * kTileDepth;
    p.splits = cdiv(k, p.k_per_split);
    if (p.splits > 1) p.bytes = align_up((size_t)p.splits * m * n * 4);
    else p.k_per_split = k;
  }
  return p;
}

bool product_fits(int64_t m, int64_t n) {
  return cdiv(m, 64) * cdiv(n, 64) <= kMaxGroups && cdiv(m * cdiv(n, 4), 256) <= kMaxGroups;
}

hipError_t run_product(ProductArgs a, const ProductPlan& p, void* ws, hipStream_t s) {
  a.splits = (int32_t)p.splits;
  a.k_per_split = p.k_per_split;
  a.partial = static_cast<float*>(ws);
  hipError_t e = launch_product_tile(a, s);
  if (e == hipSuccess && a.splits > 1) e = launch_product_finish(a, s);
  return e;
}

bool valid_act(int a) { return a >= XTVXY_ACT_NONE && a <= XTVXY_ACT_SILU; }

xtvxy_status linear_workspace(int64_t m, int64_t k, int64_t n, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || k < 0 || n < 0) return XTVXY_ERROR_INVALID_VALUE;
  if (bytes_overflow(m, n) || bytes_overflow(m, k) || bytes_overflow(n, k)) return XTVXY_ERROR_INVALID_VALUE;
  *bytes = 0;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!product_fits(m, n)) return XTVXY_ERROR_UNSUPPORTED;
  *bytes = plan_product(m, n, k).bytes;
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
  const ProductPlan plan = plan_product(m, n, k);
  if (plan.bytes > 0 && (!ws || ws_bytes < plan.bytes || reinterpret_cast<uintptr_t>(ws) % kAlign != 0))
    return XTVXY_ERROR_WORKSPACE;
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
  a.e = {bias, residual, ldr, pre, ldp, out, ldo, act,
         mo.aligned4() && (!residual || mr.aligned4()) && (!pre || mp.aligned4())};
  return status_of(run_product(a, plan, ws, stream));
}

// Workspace of the gradient: d in the element type (unless it is G itself), the column sums of the
// row groups, and the partial sums of the two products, which run one after the other.
struct BackwardPlan {
  bool form_d;
  int64_t ldd, rows_per_group, groups;
  ProductPlan dx, dw;
  size_t d_off, sums_off, partial_off, bytes;
};

BackwardPlan plan_backward(int type, int64_t m, int64_t k, int64_t n, int act) {
  BackwardPlan p{};
  p.form_d = act != XTVXY_ACT_NONE;
  p.ldd = cdiv(n, 8) * 8;
  // row groups: about four workgroups per CU, at least 32 rows each
  const int64_t column_groups = std::max<int64_t>(1, cdiv(n, 512));
  int64_t groups = std::max<int64_t>(1, 4 * kComputeUnits / column_groups);
  p.rows_per_group = std::max<int64_t>(32, cdiv(m, groups));
  p.groups = std::max<int64_t>(1, cdiv(m, p.rows_per_group));
  p.dx = plan_product(m, k, n);
  p.dw = plan_product(n, k, m);
  size_t at = 0;
  p.d_off = at;
  if (p.form_d) at += align_up((size_t)m * p.ldd * elem_size(type));
  p.sums_off = at;
  at += align_up((size_t)p.groups * n * 4);
  p.partial_off = at;
  p.bytes = at + std::max(p.dx.bytes, p.dw.bytes);
  return p;
}

bool backward_fits(int64_t m, int64_t k, int64_t n) {
  return product_fits(m, k) && product_fits(n, k) && cdiv(n, 512) <= kMaxGroups / 2048;
}

xtvxy_status backward_workspace(int type, int64_t m, int64_t k, int64_t n, int act, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || k < 0 || n < 0 || !valid_act(act)) return XTVXY_ERROR_INVALID_VALUE;
  if (bytes_overflow(m, n + 8) || bytes_overflow(m, k) || bytes_overflow(n, k)) return XTVXY_ERROR_INVALID_VALUE;
  *bytes = 0;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!backward_fits(m, k, n)) return XTVXY_ERROR_UNSUPPORTED;
  *bytes = plan_backward(type, m, k, n, act).bytes;
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

  const BackwardPlan p = plan_backward(type, m, k, n, act);
  if (reads && p.bytes > 0 && (!ws || ws_bytes < p.bytes || reinterpret_cast<uintptr_t>(ws) % kAlign != 0))
    return XTVXY_ERROR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  hipError_t e = hipSuccess;
  const void* D = G;
  int64_t ldd = ldg;
  const bool products = k > 0 && (dX || dW);
  if (reads && ((p.form_d && products) || db)) {
    SlopeArgs s{};
    s.g = G;
    s.ldg = ldg;
    s.pre = pre;
    s.ldp = ldp;
    s.d = p.form_d && products ? base + p.d_off : nullptr;
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
    if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  } else if (db && n > 0) {
    e = launch_zero(db, (size_t)n * 4, stream);
    if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  if (p.form_d) {
    D = base + p.d_off;
    ldd = p.ldd;
  }
  const Matrix md{D, m, n, ldd, es};
  if (dX && m > 0 && k > 0) {
    ProductArgs a{};
    a.A = D;
    a.lda = ldd;
    a.a_wide = md.aligned16();
    a.B = W;
    a.ldb = ldw;
    a.b_contraction_major = 1;
    a.b_wide = mw.aligned16();
    a.m = m;
    a.n = k;
    a.k = n;
    a.type = type;
    a.e = {nullptr, nullptr, 0, nullptr, 0, dX, lddx, XTVXY_ACT_NONE, mdx.aligned4()};
    e = run_product(a, p.dx, base + p.partial_off, stream);
    if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  if (dW && n > 0 && k > 0) {
    ProductArgs a{};
    a.A = D;
    a.lda = ldd;
    a.a_contraction_major = 1;
    a.a_wide = md.aligned16();
    a.B = X;
    a.ldb = ldx;
    a.b_contraction_major = 1;
    a.b_wide = mx.aligned16();
    a.m = n;
    a.n = k;
    a.k = m;
    a.type = type;
    a.e = {nullptr, nullptr, 0, nullptr, 0, dW, lddw, XTVXY_ACT_NONE, mdw.aligned4()};
    e = run_product(a, p.dw, base + p.partial_off, stream);
    if (e != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  return XTVXY_SUCCESS;
}

}  // namespace

extern "C" {

#define XTVXY_LINEAR(SUFFIX, TYPE, T)                                                                                 \
  xtvxy_status xtvxy_linear_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n, int aligned16, size_t* bytes) { \
    (void)aligned16;                                                                                                  \
    return linear_workspace(m, k, n, bytes);                                                                          \
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
    (void)aligned16;                                                                                                  \
    return backward_workspace(TYPE, m, k, n, activation, bytes);                                                      \
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
