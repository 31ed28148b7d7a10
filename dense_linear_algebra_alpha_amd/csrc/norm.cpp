// Host side of layer norm and its gradient: argument checks, workspace and launches. Argument errors are
// found before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "matrix.h"
#include "norm.h"

using namespace xtvxy;

namespace {

// What the sums of a row are made for: up to 2^17 terms of each of 1024 threads.
bool too_wide(int64_t n) { return n >= (int64_t)1 << 27; }

xtvxy_status norm_impl(int type, int64_t m, int64_t n, const void* X, int64_t ldx, const float* weight, const float* bias,
                       float eps, void* out, int64_t ldo, float* mean, float* rstd, hipStream_t stream) {
  if (m < 0 || n < 0 || !(eps >= 0.0f) || std::isinf(eps)) return XTVXY_ERROR_INVALID_VALUE;
  if (bad_ld(ldx, n, m) || bad_ld(ldo, n, m)) return XTVXY_ERROR_INVALID_VALUE;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!X || !out) return XTVXY_ERROR_NULL_POINTER;
  if (too_wide(n)) return XTVXY_ERROR_UNSUPPORTED;
  const int es = elem_size(type);
  const Matrix in[] = {{X, m, n, ldx, es}, vec(weight, n), vec(bias, n)};
  const Matrix written[] = {{out, m, n, ldo, es}, vec(mean, m), vec(rstd, m)};
  for (int o = 0; o < 3; ++o) {
    for (const Matrix& i : in)
      if (overlap(written[o], i)) return XTVXY_ERROR_ALIASING;
    for (int p = 0; p < o; ++p)
      if (overlap(written[o], written[p])) return XTVXY_ERROR_ALIASING;
  }
  return status_of(launch_norm({X, ldx, weight, bias, out, ldo, mean, rstd, m, n, eps}, type, stream));
}

xtvxy_status gradient_workspace(int64_t m, int64_t n, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || n < 0 || bytes_overflow(m, n) || n > INT64_MAX / 4096) return XTVXY_ERROR_INVALID_VALUE;
  // of either element size
  const int64_t groups = m == 0 || n == 0 ? 0 : std::max(norm_gradient_groups(m, n, kF32), norm_gradient_groups(m, n, kBf16));
  *bytes = align_up((size_t)groups * 2 * n * 4);
  return XTVXY_SUCCESS;
}

xtvxy_status gradient_impl(int type, int64_t m, int64_t n, const void* G, int64_t ldg, const void* X, int64_t ldx,
                           const float* mean, const float* rstd, const float* weight, void* dX, int64_t lddx,
                           float* dweight, float* dbias, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (m < 0 || n < 0) return XTVXY_ERROR_INVALID_VALUE;
  if (bad_ld(ldg, n, m) || bad_ld(ldx, n, m) || (dX && bad_ld(lddx, n, m))) return XTVXY_ERROR_INVALID_VALUE;
  const bool sums = dweight || dbias;
  if (n == 0 || (!dX && !sums)) return XTVXY_SUCCESS;
  if (m > 0 && (!G || !X || !mean || !rstd)) return XTVXY_ERROR_NULL_POINTER;
  if (too_wide(n)) return XTVXY_ERROR_UNSUPPORTED;
  const int es = elem_size(type);
  const Matrix in[] = {{G, m, n, ldg, es}, {X, m, n, ldx, es}, vec(mean, m), vec(rstd, m), vec(weight, n)};
  const Matrix written[] = {{dX, m, n, lddx, es}, vec(dweight, n), vec(dbias, n)};
  for (int o = 0; o < 3; ++o) {
    for (const Matrix& i : in)
      if (overlap(written[o], i)) return XTVXY_ERROR_ALIASING;
    for (int p = 0; p < o; ++p)
      if (overlap(written[o], written[p])) return XTVXY_ERROR_ALIASING;
  }
  if (m == 0) {  // empty sums
    if (dweight && launch_zero(dweight, (size_t)n * 4, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    return status_of(dbias ? launch_zero(dbias, (size_t)n * 4, stream) : hipSuccess);
  }
  const int64_t groups = norm_gradient_groups(m, n, type);
  const size_t need = sums ? align_up((size_t)groups * 2 * n * 4) : 0;
  if (need > 0 && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % kAlign != 0)) return XTVXY_ERROR_WORKSPACE;
  return status_of(launch_norm_gradient({G, X, mean, rstd, weight, dX, ldg, ldx, lddx, m, n,
                                         sums ? static_cast<float*>(ws) : nullptr, groups, dweight, dbias}, type, stream));
}

}  // namespace

extern "C" {

xtvxy_status xtvxy_layer_norm_backward_workspace_size(int64_t m, int64_t n, size_t* bytes) {
  return gradient_workspace(m, n, bytes);
}

#define XTVXY_LAYER_NORM(SUFFIX, TYPE, T)                                                                              \
  xtvxy_status xtvxy_layer_norm_##SUFFIX(int64_t m, int64_t n, const T* X, int64_t ldx, const float* weight,           \
                                         const float* bias, float eps, T* out, int64_t ldo, float* mean, float* rstd,  \
                                         hipStream_t stream) {                                                         \
    return norm_impl(TYPE, m, n, X, ldx, weight, bias, eps, out, ldo, mean, rstd, stream);                             \
  }                                                                                                                    \
  xtvxy_status xtvxy_layer_norm_backward_##SUFFIX(int64_t m, int64_t n, const T* G, int64_t ldg, const T* X,           \
                                                  int64_t ldx, const float* mean, const float* rstd,                   \
                                                  const float* weight, T* dX, int64_t lddx, float* dweight,            \
                                                  float* dbias, void* workspace, size_t workspace_bytes,               \
                                                  hipStream_t stream) {                                                \
    return gradient_impl(TYPE, m, n, G, ldg, X, ldx, mean, rstd, weight, dX, lddx, dweight, dbias, workspace,          \
                         workspace_bytes, stream);                                                                     \
  }

XTVXY_LAYER_NORM(f32, kF32, float)
XTVXY_LAYER_NORM(bf16, kBf16, uint16_t)
XTVXY_LAYER_NORM(f16, kF16, uint16_t)

}  // extern "C"
