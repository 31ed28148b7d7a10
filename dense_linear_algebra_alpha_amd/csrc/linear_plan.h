// How products are planned: the kernel, tile and parts of each, and the copies of matrices whose rows do not suit.
// Shared by the layer (linear.cpp) and the losses over an output layer (loss.cpp).
#pragma once

#include "linear.h"
#include "matrix.h"

namespace xtvxy {

constexpr int64_t kComputeUnits = 256;           // the plans are for this chip whatever runs the query
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads in one launch: below 2^32 threads

// How one product is computed: by which kernel, which of its tiles whole and which in how many parts of
// the contraction.
struct ProductPlan {
  int tile = 0;  // 0: the kernel for any alignment; 64, 128, 256: the ring kernel's tile
  int64_t whole = 0, splits = 1, k_per_split = 0;
  size_t bytes = 0;  // partial sums
  double us = 0;     // estimated time of the launch (of a gradient's two products together)
};

// Plans of the shapes of a thread's latest calls. The search takes 1.2 us for a layer (15 at most over 600 shapes)
// and 8 for a gradient (26), and a gradient's workspace query looks at up to 24 of them; a call takes 4.
template <typename Plan>
struct PlanCache {
  struct Entry {
    int64_t key[4] = {-1, -1, -1, -1};
    Plan plan{};
  } entries[64];
  template <typename Make>
  const Plan& get(int64_t m, int64_t k, int64_t n, int64_t what, Make make) {
    const uint64_t h = (uint64_t)m * 0x9E3779B97F4A7C15u ^ (uint64_t)k * 0xC2B2AE3D27D4EB4Fu ^ (uint64_t)n * 0x165667B19E3779F9u ^
                       (uint64_t)what * 0x27D4EB2F165667C5u;
    Entry& e = entries[(h >> 40) % 64];
    const int64_t key[4] = {m, k, n, what};
    if (!std::equal(key, key + 4, e.key)) {
      e.plan = make();
      std::copy(key, key + 4, e.key);
    }
    return e.plan;
  }
};

inline bool product_fits(int64_t m, int64_t n) {
  return cdiv(m, 64) * cdiv(n, 64) <= kMaxGroups;
}

inline bool backward_fits(int64_t m, int64_t k, int64_t n) {
  // both products are one launch
  return cdiv(m, 64) * cdiv(k, 64) + cdiv(n, 64) * cdiv(k, 64) + cdiv(n, 16) <= kMaxGroups;
}

inline void take_plan(ProductArgs* a, const ProductPlan& p, void* ws) {
  a->tile = p.tile;
  a->whole = p.tile ? p.whole : 0;
  a->splits = (int32_t)p.splits;
  a->k_per_split = p.k_per_split;
  a->partial = static_cast<float*>(ws);
}

inline int64_t padded(int64_t cols, int es) { return cdiv(cols, 16 / es) * (16 / es); }

inline bool whole_chunks(const Matrix& x) {
  return x.aligned16() && x.cols * x.es % 16 == 0 && x.ld * x.es <= kRingMaxPitch;
}

inline size_t packed_bytes(int64_t rows, int64_t cols, int es) { return align_up((size_t)rows * padded(cols, es) * es); }

// The kernel for few rows: its wavefronts (0: not for this shape), outputs of a workgroup, and parts.
struct FewPlan {
  int waves = 0, outputs = 0;
  ProductPlan product;
};
FewPlan plan_few(int type, int64_t m, int64_t k, int64_t n);
// The layer's tile, split tiles and parts with the least estimated time; without `split` no tile is split. only_tile:
// that tile, if not 0.
ProductPlan plan_product(int type, int64_t m, int64_t n, int64_t k, bool ring, bool split = true, int only_tile = 0);
// The same for the gradient's products dX (m x k, contraction n) and dW (n x k, contraction m), which share a tile
// and a launch. dx_in_parts: dX's tiles are split alike (whole 0).
void plan_gradient(int type, int64_t m, int64_t k, int64_t n, bool want_dx, bool want_dw, bool ring, ProductPlan* dx,
                   ProductPlan* dw, int only_tile = 0, bool dx_in_parts = false);

}  // namespace xtvxy
