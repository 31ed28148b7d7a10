// Internal declarations of the embedding lookup and its gradient (embedding.cpp, embedding.hip).
#pragma once

#include "linear.h"

namespace xtvxy {

struct EmbeddingArgs {
  const void* ids;
  int32_t index_bits;
  int64_t count, k, rows;
  const void* table;
  int64_t ldt;
  float scale;
  void* out;
  int64_t ldo;
};
hipError_t launch_embedding(const EmbeddingArgs& a, int type, hipStream_t s);

constexpr int kSortItems = 16384;    // keys of a sorting workgroup (1024 threads x 16)
constexpr int kDigitBits = 9;        // most bits of a sorting pass
constexpr int kDigits = 1 << kDigitBits;
constexpr int kPieceTokens = 32;     // sorted tokens that a wavefront sums
constexpr int kSlabBytes = 1024;     // of a row's columns, per wavefront

struct EmbeddingGradientArgs {
  const void* g;
  int64_t ldg;
  const void* ids;
  int32_t index_bits, accumulate;
  int64_t count, k, rows;
  float scale;
  void* dtable;
  int64_t lddt;
  // workspace: tokens sorted by their row (keys; rows: no row) and where they come from, twice where
  // several workgroups sort; counts[sorting workgroups][kDigits]; the sums of rows that cross pieces
  uint32_t* keys[2];
  uint32_t* from[2];
  uint32_t* counts;
  float* partial;       // [pieces][2][padded columns]
};
inline int64_t sort_groups(int64_t count) { return (count + kSortItems - 1) / kSortItems; }
inline int64_t piece_count(int64_t count) { return (count + kPieceTokens - 1) / kPieceTokens; }
inline int64_t slab_columns(int type) { return kSlabBytes / elem_size(type); }
hipError_t launch_embedding_gradient(const EmbeddingGradientArgs& a, int type, hipStream_t s);

}  // namespace xtvxy
