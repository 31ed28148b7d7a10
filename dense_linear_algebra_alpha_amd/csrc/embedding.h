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

constexpr int kSortAlone = 4096;        // keys up to which one workgroup sorts
constexpr int kSortUncounted = 32768;   // up to which its passes do without a launch that counts digits
constexpr int kCountedTile = 4096;      // keys of a workgroup beyond (1024 up to there)
constexpr int kDigitBits = 9;        // most bits of their passes
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSlabBytes = 1024;     // of a row's columns, per wavefront

struct EmbeddingGradientArgs {
  const void* g;
  int64_t ldg;
  const void* ids;
  int32_t index_bits, accumulate;
  int64_t count, k, rows;
  float scale;
  int32_t piece;        // tokens
  void* dtable;
  int64_t lddt;
  // workspace: tokens sorted by their row (keys; rows: no row) and where they come from, twice where
  // several workgroups sort; counts[sorting workgroups][kDigits]; the sums of rows that cross pieces
  uint32_t* keys[2];
  uint32_t* from[2];
  uint32_t* counts;
  float* partial;       // [pieces][2][padded columns]
};
inline int64_t sort_groups(int64_t count) { return count <= kSortAlone ? (count > 0) : count <= kSortUncounted ? (count + 1023) / 1024 : (count + kCountedTile - 1) / kCountedTile; }
inline int64_t slab_columns(int type) { return kSlabBytes / elem_size(type); }
// Sorted tokens that a wavefront sums: 32, or fewer where that leaves CUs without work (a wavefront loads 8 rows at a
// time, and each time waits for memory). us with 8, 16 and 32: 4000 tokens of two slabs 24, 26, 32; 8000 of two 32, 33, 39;
// 40000 of one 56, 52, 55; 16384 of four 80, 75, 76; 65536 of two 106, 98, 92.
inline int piece_tokens(int64_t count, int64_t slabs) { return count * slabs >= 96 * 1024 ? 32 : count * slabs >= 24 * 1024 ? 16 : 8; }
inline int64_t piece_count(int64_t count, int piece) { return (count + piece - 1) / piece; }
hipError_t launch_embedding_gradient(const EmbeddingGradientArgs& a, int type, hipStream_t s);

}  // namespace xtvxy
