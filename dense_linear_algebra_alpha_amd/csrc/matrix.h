// Host-side checks that the entry points on matrices share: sizes, strides, overlaps.
#pragma once

#include <algorithm>
#include <cstdint>

#include "internal.h"

namespace xtvxy {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool bytes_overflow(int64_t rows, int64_t ld) { return rows > 0 && ld > INT64_MAX / 16 / rows; }
// The same for rows of cols elements padded by up to 8.
inline bool padded_overflow(int64_t rows, int64_t cols) { return rows > 0 && cols > INT64_MAX / 16 / rows - 8; }

struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
  int es;
  size_t extent() const { return rows > 0 && cols > 0 ? (size_t)((rows - 1) * ld + cols) * es : 0; }
  bool aligned16() const { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0; }
};

// Whether two matrices share an element (rows of equal pitch: exact; else by their extents).
inline bool overlap(const Matrix& a, const Matrix& b) {
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

inline Matrix vec(const float* p, int64_t n) { return {p, 1, n, n > 0 ? n : 1, 4}; }

inline bool bad_ld(int64_t ld, int64_t cols, int64_t rows) { return ld < std::max<int64_t>(cols, 1) || bytes_overflow(rows, ld); }

inline xtvxy_status status_of(hipError_t e) { return e == hipSuccess ? XTVXY_SUCCESS : XTVXY_ERROR_LAUNCH; }

}  // namespace xtvxy
