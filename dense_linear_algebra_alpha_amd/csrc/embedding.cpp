// Host side of the embedding lookup and its gradient: argument checks, workspace and launches. Argument
// errors are found before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "embedding.h"
#include "matrix.h"

using namespace xtvxy;

namespace {

constexpr int64_t kMostTokens = (int64_t)1 << 26;  // a sorting workgroup reads the counts of all others
constexpr int64_t kMostRows = INT32_MAX - 1;

Matrix indices(const void* p, int64_t n, int bits) { return {p, 1, n, n > 0 ? n : 1, bits / 8}; }

xtvxy_status embedding_impl(int type, int64_t count, int64_t k, int64_t rows, const void* ids, int index_bits,
                            const void* table, int64_t ldt, float scale, void* out, int64_t ldo, hipStream_t stream) {
  if (count < 0 || k < 0 || rows < 0 || (index_bits != 32 && index_bits != 64)) return XTVXY_ERROR_INVALID_VALUE;
  if (bad_ld(ldt, k, rows) || bad_ld(ldo, k, count)) return XTVXY_ERROR_INVALID_VALUE;
  if (count == 0 || k == 0) return XTVXY_SUCCESS;
  if (!ids || !out || (rows > 0 && !table)) return XTVXY_ERROR_NULL_POINTER;
  const int es = elem_size(type);
  const Matrix mo{out, count, k, ldo, es}, mt{table, rows, k, ldt, es};
  if (overlap(mo, mt) || overlap(mo, indices(ids, count, index_bits))) return XTVXY_ERROR_ALIASING;
  return status_of(launch_embedding({ids, index_bits, count, k, rows, table, ldt, scale, out, ldo}, type, stream));
}

struct GradientPlan {
  int piece = 0;
  size_t keys[2], from[2], counts, partial, bytes = 0;
};

GradientPlan plan_gradient(int type, int64_t count, int64_t k) {
  GradientPlan p;
  const auto take = [&](size_t bytes) {
    const size_t at = p.bytes;
    p.bytes += align_up(bytes);
    return at;
  };
  const int64_t groups = sort_groups(count);
  for (int i = 0; i < 2; ++i) {  // one workgroup sorts in LDS: no second copy
    p.keys[i] = take(i == 0 || groups > 1 ? (size_t)count * 4 : 0);
    p.from[i] = take(i == 0 || groups > 1 ? (size_t)count * 4 : 0);
  }
  p.counts = take(count > kSortUncounted ? (size_t)groups * kDigits * 4 : 0);
  const int64_t columns = slab_columns(type);
  p.piece = piece_tokens(count, cdiv(k, columns));
  const int64_t pieces = piece_count(count, p.piece);
  p.partial = take(pieces > 1 ? (size_t)pieces * 2 * (cdiv(k, columns) * columns) * 4 : 0);
  return p;
}

xtvxy_status gradient_limits(int type, int64_t count, int64_t k, int64_t rows) {
  if (count < 0 || k < 0 || rows < 0 || padded_overflow(count, k) || bytes_overflow(rows, k)) return XTVXY_ERROR_INVALID_VALUE;
  // pieces x slabs are one launch's workgroups
  const int64_t slabs = cdiv(k, slab_columns(type));
  if (count > kMostTokens || rows > kMostRows || (slabs > 0 && piece_count(count, 32) > (((int64_t)1 << 24) - 1) / slabs))
    return XTVXY_ERROR_UNSUPPORTED;
  return XTVXY_SUCCESS;
}

xtvxy_status gradient_workspace(int type, int64_t count, int64_t k, int64_t rows, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  const xtvxy_status st = gradient_limits(type, count, k, rows);
  if (st != XTVXY_SUCCESS) return st;
  *bytes = count == 0 || k == 0 || rows == 0 ? 0 : plan_gradient(type, count, k).bytes;
  return XTVXY_SUCCESS;
}

xtvxy_status gradient_impl(int type, int64_t count, int64_t k, int64_t rows, const void* G, int64_t ldg, const void* ids,
                           int index_bits, float scale, int accumulate, void* dtable, int64_t lddt, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  if (index_bits != 32 && index_bits != 64) return XTVXY_ERROR_INVALID_VALUE;
  const xtvxy_status st = gradient_limits(type, count, k, rows);
  if (st != XTVXY_SUCCESS) return st;
  if (bad_ld(ldg, k, count) || bad_ld(lddt, k, rows)) return XTVXY_ERROR_INVALID_VALUE;
  if (k == 0 || rows == 0) return XTVXY_SUCCESS;
  if (!dtable || (count > 0 && (!G || !ids))) return XTVXY_ERROR_NULL_POINTER;
  const int es = elem_size(type);
  const Matrix mo{dtable, rows, k, lddt, es}, mg{G, count, k, ldg, es};
  if (overlap(mo, mg) || overlap(mo, indices(ids, count, index_bits))) return XTVXY_ERROR_ALIASING;
  const GradientPlan p = count > 0 ? plan_gradient(type, count, k) : GradientPlan{};
  if (count > 0 && (!ws || ws_bytes < p.bytes || reinterpret_cast<uintptr_t>(ws) % kAlign != 0)) return XTVXY_ERROR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  EmbeddingGradientArgs a{G, ldg, ids, index_bits, accumulate != 0, count, k, rows, scale, p.piece, dtable, lddt, {}, {}, nullptr, nullptr};
  if (count > 0) {
    for (int i = 0; i < 2; ++i) {
      a.keys[i] = reinterpret_cast<uint32_t*>(base + p.keys[i]);
      a.from[i] = reinterpret_cast<uint32_t*>(base + p.from[i]);
    }
    a.counts = reinterpret_cast<uint32_t*>(base + p.counts);
    a.partial = reinterpret_cast<float*>(base + p.partial);
  }
  return status_of(launch_embedding_gradient(a, type, stream));
}

}  // namespace

extern "C" {

#define XTVXY_EMBEDDING(SUFFIX, TYPE, T)                                                                               \
  xtvxy_status xtvxy_embedding_##SUFFIX(int64_t count, int64_t k, int64_t rows, const void* ids, int index_bits,       \
                                        const T* table, int64_t ldt, float scale, T* out, int64_t ldo,                 \
                                        hipStream_t stream) {                                                          \
    return embedding_impl(TYPE, count, k, rows, ids, index_bits, table, ldt, scale, out, ldo, stream);                 \
  }                                                                                                                    \
  xtvxy_status xtvxy_embedding_backward_##SUFFIX##_workspace_size(int64_t count, int64_t k, int64_t rows,              \
                                                                  size_t* bytes) {                                     \
    return gradient_workspace(TYPE, count, k, rows, bytes);                                                            \
  }                                                                                                                    \
  xtvxy_status xtvxy_embedding_backward_##SUFFIX(int64_t count, int64_t k, int64_t rows, const T* G, int64_t ldg,      \
                                                 const void* ids, int index_bits, float scale, int accumulate,         \
                                                 T* dtable, int64_t lddt, void* workspace, size_t workspace_bytes,     \
                                                 hipStream_t stream) {                                                 \
    return gradient_impl(TYPE, count, k, rows, G, ldg, ids, index_bits, scale, accumulate, dtable, lddt, workspace,    \
                         workspace_bytes, stream);                                                                     \
  }

XTVXY_EMBEDDING(f32, kF32, float)
XTVXY_EMBEDDING(bf16, kBf16, uint16_t)
XTVXY_EMBEDDING(f16, kF16, uint16_t)

}  // extern "C"
