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
// The same for rows of cols elements padded by up to 8.
bool padded_overflow(int64_t rows, int64_t cols) { return rows > 0 && cols > INT64_MAX / 16 / rows - 8; }

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

// How one product is computed: by which kernel, which of its tiles whole and which in how many parts of
// the contraction.
struct ProductPlan {
  int tile = 0;  // 0: the kernel for any alignment; 64, 128, 256: the ring kernel's tile
  int64_t whole = 0, splits = 1, k_per_split = 0;
  size_t bytes = 0;  // partial sums
};

// The estimate of a launch's time. Its workgroups are jobs of so many stages (32 steps; fp32: 16). A CU
// holds one of 256 x 256, two of 128 x 128 or five of 64 x 64 at a time, and works off a stage in
// stage_us of the matrix unit and LDS; a smaller tile alone on its CU waits instead, alone_us a stage.
// The constants were fitted to 1842 measured choices of tile and parts for 62 products and gradients of
// 2^23 to 2^36 multiplications: what the estimate picks is 1.0% slower than the best one in the geometric
// mean, 12% at most (one tile for all: 256 x 256 up to 3.2 times slower, 128 x 128 2.0, 64 x 64 2.6).
int residents(int tile) { return tile == 256 ? 1 : tile == 128 ? 2 : 5; }
double stage_us(int type, int tile) {
  if (type == kF32) return tile == 128 ? 1.12 : 0.28;
  return tile == 256 ? 0.70 : tile == 128 ? 0.27 : 0.125;
}
double alone_us(int type, int tile) {
  if (type == kF32) return tile == 128 ? 1.15 : 0.36;
  return tile == 256 ? 0.70 : tile == 128 ? 0.33 : 0.18;
}
// First loads and epilogue; those of a CU's further workgroups are hidden but for next_us.
double ends_us(int tile) { return tile == 256 ? 9.0 : tile == 128 ? 4.5 : 5.5; }
double next_us(int tile) { return tile == 128 ? 1.5 : 0.7; }
// A split: the launch that sums the parts, their sums written and read back.
constexpr double kFinishUs = 8.0, kPartsBytesPerUs = 4e6;

struct Jobs {
  int64_t count = 0, stages = 0;
};
// When the last of the jobs ends, each in turn given to the CU that is free first.
double makespan(const Jobs* jobs, int kinds, double us_per_stage, double us_per_job) {
  struct Class {  // CUs that are free from the same time on
    double at;
    int64_t count;
  } free_at[8] = {{0.0, kComputeUnits}};
  int classes = 1;
  double last = 0;
  for (int j = 0; j < kinds; ++j) {
    int64_t left = jobs[j].count;
    while (left > 0) {
      int first = 0;
      for (int c = 1; c < classes; ++c)
        if (free_at[c].at < free_at[first].at) first = c;
      const int64_t rounds = classes == 1 ? std::max<int64_t>(1, left / free_at[first].count) : 1;
      const int64_t n = std::min(left, free_at[first].count * rounds);
      const double end = free_at[first].at + rounds * (jobs[j].stages * us_per_stage + us_per_job);
      left -= n;
      last = std::max(last, end);
      const int64_t used = std::min(n, free_at[first].count);
      if ((free_at[first].count -= used) == 0) free_at[first] = free_at[--classes];
      int same = 0;
      while (same < classes && free_at[same].at != end) ++same;
      if (same < classes) free_at[same].count += used;
      else free_at[classes++] = {end, used};  // at most one class more per kind of job
    }
  }
  return last;
}

// When the last of the jobs ends where CUs share themselves among several.
double shared_end(int type, int tile, const Jobs* jobs, int kinds) {
  const double us = stage_us(type, tile), ends = ends_us(tile);
  int64_t total = 0, stages = 0, longest = 0, last = 0, upto[5] = {0};
  for (int j = 0; j < kinds; ++j) {
    total += jobs[j].count;
    stages += jobs[j].count * jobs[j].stages;
    upto[j + 1] = total;
    if (jobs[j].count > 0) longest = std::max(longest, last = jobs[j].stages);
  }
  if (total > kComputeUnits * residents(tile)) {
    // later jobs go where there is room, so the loads are even but for the last jobs; a job that is longer
    // than its CU's load goes on alone
    const double load = stages * us / kComputeUnits, all = us * residents(tile);
    const double even = load + 0.3 * last * all + next_us(tile) * ((double)total / kComputeUnits - 1);
    return std::max(even, load + (longest - load / all) * alone_us(type, tile)) + ends;
  }
  // the epilogue of a lone 128 x 128 tile is on nobody's cover
  double latest = longest * alone_us(type, tile) + ends + (tile == 128 && total <= kComputeUnits ? 2.0 : 0.0);
  for (int b = 0; b < 2 * kinds + 2; ++b) {  // the CUs in turn: the loads change where a kind of job ends
    const int64_t cu = (upto[b / 2] + kComputeUnits - b % 2) % kComputeUnits;
    int64_t load = 0, held = 0;
    for (int j = 0; j < kinds; ++j) {
      const auto before = [&](int64_t n) { return n > cu ? (n - cu + kComputeUnits - 1) / kComputeUnits : 0; };
      const int64_t mine = before(upto[j + 1]) - before(upto[j]);
      load += mine * jobs[j].stages;
      held += mine;
    }
    latest = std::max(latest, load * us + ends + next_us(tile) * std::max<int64_t>(0, held - 1));
  }
  return latest;
}

double launch_us(int type, int tile, const Jobs* jobs, int kinds) {
  return tile == 256 ? makespan(jobs, kinds, stage_us(type, tile), ends_us(tile)) : shared_end(type, tile, jobs, kinds);
}

constexpr int64_t kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
constexpr int64_t kMostParts = 5 * kComputeUnits;  // workgroups of split tiles

// A product with a tile, `whole` of its tiles not split. False where the split makes no sense.
bool set_product(ProductPlan* p, int type, int tile, bool ring, int64_t whole, int64_t splits, int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = cdiv(m, tile) * cdiv(n, tile);
  p->tile = ring ? tile : 0;
  p->splits = splits;
  p->whole = splits > 1 ? whole : tiles;
  p->k_per_split = std::max<int64_t>(kTileDepth, cdiv(cdiv(k, splits), kTileDepth) * kTileDepth);
  p->bytes = splits == 1 ? 0 : align_up((size_t)splits * (ring ? (tiles - whole) * tile * tile : m * n) * 4);
  return splits == 1 || (p->k_per_split >= 64 && (tiles - whole) * splits <= kMostParts && cdiv(k, p->k_per_split) == splits);
}

// The jobs of a product; returns the time of its parts' sums.
double product_jobs(const ProductPlan& p, int type, int tile, int64_t m, int64_t n, int64_t k, Jobs* jobs) {
  const int64_t tiles = cdiv(m, tile) * cdiv(n, tile), whole = p.splits > 1 ? p.whole : tiles;
  const int64_t depth = type == kF32 ? 16 : 32;
  jobs[0] = {whole, cdiv(k, depth)};
  jobs[1] = {(tiles - whole) * p.splits, cdiv(p.k_per_split, depth)};
  return p.splits > 1 ? 2.0 * p.splits * (tiles - whole) * tile * tile * 4 / kPartsBytesPerUs : 0.0;
}

// The layer's tile, split tiles and parts with the least estimated time.
ProductPlan plan_product(int type, int64_t m, int64_t n, int64_t k, bool ring) {
  ProductPlan best;
  best.k_per_split = kTileDepth;
  if (m == 0 || n == 0) return best;
  double least = 0;
  for (int tile : {64, 128, 256}) {
    if (!ring ? tile != 64 : (tile == 256 && type == kF32)) continue;
    const int64_t tiles = cdiv(m, tile) * cdiv(n, tile), slots = kComputeUnits * residents(tile);
    // what a last, incomplete round of the CUs would hold may be split instead of everything
    const int64_t whole[] = {0, tiles / kComputeUnits * kComputeUnits, tiles / slots * slots};
    for (int w = 0; w < (ring ? 3 : 1); ++w) {
      if (w > 0 && (whole[w] == 0 || whole[w] == tiles)) continue;
      for (int64_t splits : kSplits) {
        ProductPlan p;
        if ((w > 0 && splits == 1) || !set_product(&p, type, tile, ring, whole[w], splits, m, n, k)) continue;
        if (splits > 1 && tiles + kMostParts > kMaxGroups) continue;  // beyond one launch
        Jobs jobs[2];
        double us = product_jobs(p, type, tile, m, n, k, jobs) + (splits > 1 ? kFinishUs : 0.0);
        us += launch_us(type, tile, jobs, 2);
        if (least == 0 || us < least) {
          least = us;
          best = p;
        }
      }
    }
  }
  return best;
}

// The gradient's products dX (m x k, contraction n) and dW (n x k, contraction m) share a tile and a
// launch, the one with the longer contraction first.
void plan_gradient(int type, int64_t m, int64_t k, int64_t n, bool want_dx, bool want_dw, bool ring, ProductPlan* dx,
                   ProductPlan* dw) {
  dx->k_per_split = dw->k_per_split = kTileDepth;
  if (m == 0 || k == 0 || n == 0) return;
  const bool dw_first = m > n;
  double least = 0;
  for (int tile : {64, 128, 256}) {
    if (!ring ? tile != 64 : (tile == 256 && type == kF32)) continue;
    const int64_t tx = want_dx ? cdiv(m, tile) * cdiv(k, tile) : 0, tw = want_dw ? cdiv(n, tile) * cdiv(k, tile) : 0;
    // of the product that runs last, those tiles that its last, incomplete round would hold
    const int64_t last = dw_first ? tx : tw, full = (tx + tw) / kComputeUnits * kComputeUnits - (tx + tw - last);
    for (int rest = 0; rest < (ring && full > 0 && full < last ? 2 : 1); ++rest)
      for (int64_t sx : kSplits) {
        ProductPlan px, pw;
        if (!want_dx ? sx > 1 : !set_product(&px, type, tile, ring, rest && dw_first ? full : 0, sx, m, k, n)) continue;
        for (int64_t sw : kSplits) {
          if (rest && (dw_first ? sx : sw) == 1) continue;
          if (!want_dw ? sw > 1 : !set_product(&pw, type, tile, ring, rest && !dw_first ? full : 0, sw, n, k, m)) continue;
          if ((sx > 1 || sw > 1) && tx + tw + cdiv(n, 16) + 2 * kMostParts > kMaxGroups) continue;
          Jobs jobs[4];
          double us = sx > 1 || sw > 1 ? kFinishUs : 0.0;
          if (want_dx) us += product_jobs(px, type, tile, m, k, n, jobs + (dw_first ? 2 : 0));
          if (want_dw) us += product_jobs(pw, type, tile, n, k, m, jobs + (dw_first ? 0 : 2));
          us += launch_us(type, tile, jobs, 4);
          if (least == 0 || us < least) {
            least = us;
            *dx = want_dx ? px : ProductPlan{};
            *dw = want_dw ? pw : ProductPlan{};
          }
        }
      }
  }
}

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

bool product_fits(int64_t m, int64_t n) {
  return cdiv(m, 64) * cdiv(n, 64) <= kMaxGroups;
}

void take_plan(ProductArgs* a, const ProductPlan& p, void* ws) {
  a->tile = p.tile;
  a->whole = p.tile ? p.whole : 0;
  a->splits = (int32_t)p.splits;
  a->k_per_split = p.k_per_split;
  a->partial = static_cast<float*>(ws);
}

hipError_t run_layer(ProductArgs a, const ProductPlan& p, void* ws, hipStream_t s) {
  take_plan(&a, p, ws);
  hipError_t e = p.tile ? launch_layer_ring(a, s) : launch_layer_tile(a, s);
  if (e == hipSuccess && a.splits > 1) e = launch_product_finish(a, s);
  return e;
}

// A product's operand as the ring kernel takes it: the caller's matrix where its rows are 16-byte
// aligned and whole 16-byte chunks, else a copy in the workspace with rows padded by zeros. Small
// products take any operand as it is. us, direct against copied, fp16: 300 x 301 x 303 7.5, 10.1;
// 100 x 5001 x 900 12.6, 18.6; 1023 x 1111 x 777 13.3, 15.6; 2000 x 1001 x 1000 18.2, 21.3;
// 2000 x 501 x 3001 28.4, 32.0; 2000 x 2001 x 2001 43.3, 43.7; 4000 x 2001 x 4000 80, 79; fp32 at the last
// four 45, 47; 64, 64; 140, 137; 520, 507.
constexpr int64_t kSmallProduct = (int64_t)1 << 33;  // multiplications
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

LinearPlan make_linear_plan(int type, int64_t m, int64_t k, int64_t n, bool x_whole, bool w_whole) {
  LinearPlan p;
  const int es = elem_size(type);
  if (m <= kFewRows) {
    // W cold, us: 16 outputs a workgroup against 32: 1 x 4096 x 4096 bf16 8.9, 11.9; 13 x 2048 x 8192 11.2, 10.5
    // (X is loaded once per workgroup); 20 x 8192 x 14336 74, 60; but where 32 leave more CUs without work in
    // the last round 12 x 8192 x 10000 45, 50, 6 x 7296 x 9958 fp32 70, 79. 4 wavefronts against 8: bf16 8.9, 9.5,
    // fp32 18.1, 16.9. The ring kernel with its best split: 13.9, 14.8, 13.9, 27.4, 13.2, 15.4; at 32 rows of
    // 4096 x 4096 15.6 against 14.7, at 48 14.9 against 21.
    const auto busy = [](int64_t groups) { return (double)groups / (cdiv(groups, kComputeUnits) * kComputeUnits); };
    const bool wide = m > 4 && n >= 8192 && 1.15 * busy(cdiv(n, 32)) >= busy(cdiv(n, 16));
    const int outputs = wide ? 32 : 16;
    const int64_t groups = cdiv(n, outputs);
    const int waves = k >= 4096 && (type == kF32 || groups < kComputeUnits) ? 8 : 4;
    if (groups * (waves / 4) <= kMaxGroups) {  // else the kernels below, whose workgroups take 64 outputs or more
      p.few = waves;
      p.few_outputs = outputs;
      // Where the outputs are too few for the CUs the contraction is split, into the fewest parts that keep them
      // busy: 1 x 8192 x 1024 12.1 to 9.7, 1 x 16384 x 256 20.1 to 9.0, 23 x 11392 x 2528 (158 groups) 30.1 in one part,
      // 33.3 in two, 25.7 in three; 9 x 10368 x 3046 fp32 (191 groups) 38 in one part, 42 in two.
      int64_t splits = 1;
      if (groups < kComputeUnits && busy(groups) < 0.7 && k * es >= 16384) {
        const int64_t most = std::max<int64_t>(1, std::min<int64_t>(8, k / (waves * 256)));
        for (int64_t s = 2; s <= most && busy(groups * splits) < 0.9; ++s)
          if (busy(groups * s) > busy(groups * splits)) splits = s;
      }
      p.product.k_per_split = std::max<int64_t>(32, cdiv(cdiv(k, waves * splits), 32) * 32);
      p.product.splits = std::max<int64_t>(1, cdiv(k, waves * p.product.k_per_split));
      if (p.product.splits > 1) p.bytes = p.product.bytes = align_up((size_t)p.product.splits * m * n * 4);
      return p;
    }
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

const LinearPlan& plan_linear(int type, int64_t m, int64_t k, int64_t n, bool x_whole, bool w_whole) {
  thread_local PlanCache<LinearPlan> cache;
  return cache.get(m, k, n, type * 4 + x_whole * 2 + w_whole, [&] { return make_linear_plan(type, m, k, n, x_whole, w_whole); });
}

xtvxy_status linear_workspace(int type, int64_t m, int64_t k, int64_t n, int aligned16, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || k < 0 || n < 0) return XTVXY_ERROR_INVALID_VALUE;
  if (bytes_overflow(m, n) || padded_overflow(m, k) || padded_overflow(n, k)) return XTVXY_ERROR_INVALID_VALUE;
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
  const LinearPlan& plan = plan_linear(type, m, k, n, whole_chunks(mx), whole_chunks(mw));
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

BackwardPlan make_backward_plan(int type, int64_t m, int64_t k, int64_t n, int act, bool g_whole, bool x_whole, bool w_whole,
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
  struct Products {
    ProductPlan dx, dw;
  };
  thread_local PlanCache<Products> cache;  // the search does not depend on the matrices' alignment
  const Products& products = cache.get(m, k, n, type * 8 + want_dx * 4 + want_dw * 2 + ring, [&] {
    Products both;
    plan_gradient(type, m, k, n, want_dx, want_dw, ring, &both.dx, &both.dw);
    return both;
  });
  p.dx = products.dx;
  p.dw = products.dw;
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

const BackwardPlan& plan_backward(int type, int64_t m, int64_t k, int64_t n, int act, bool g_whole, bool x_whole,
                                  bool w_whole, bool want_dx, bool want_dw) {
  thread_local PlanCache<BackwardPlan> cache;
  const int64_t what = (((((type * 8 + act) * 2 + g_whole) * 2 + x_whole) * 2 + w_whole) * 2 + want_dx) * 2 + want_dw;
  return cache.get(m, k, n, what, [&] {
    return make_backward_plan(type, m, k, n, act, g_whole, x_whole, w_whole, want_dx, want_dw);
  });
}

bool backward_fits(int64_t m, int64_t k, int64_t n) {
  // both products are one launch
  return cdiv(m, 64) * cdiv(k, 64) + cdiv(n, 64) * cdiv(k, 64) + cdiv(n, 16) <= kMaxGroups;
}

size_t most_backward_bytes(int type, int64_t m, int64_t k, int64_t n, int act, int aligned16) {
  size_t bytes = 0;
  const int es = elem_size(type);
  const bool kc = k * es % 16 == 0, nc = n * es % 16 == 0;
  for (int c = 0; c < 8; ++c) {
    const bool g = c & 1, x = c & 2, w = c & 4;
    if (aligned16 && !(g == nc && x == kc && w == kc)) continue;
    // a product alone may be split further than the two together
    for (int want = 1; want < 4; ++want)
      bytes = std::max(bytes, make_backward_plan(type, m, k, n, act, nc && g, kc && x, kc && w, want & 1, want & 2).bytes);
  }
  return bytes;
}

xtvxy_status backward_workspace(int type, int64_t m, int64_t k, int64_t n, int act, int aligned16, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  if (m < 0 || k < 0 || n < 0 || !valid_act(act)) return XTVXY_ERROR_INVALID_VALUE;
  if (padded_overflow(m, n) || padded_overflow(m, k) || padded_overflow(n, k)) return XTVXY_ERROR_INVALID_VALUE;
  *bytes = 0;
  if (m == 0 || n == 0) return XTVXY_SUCCESS;
  if (!backward_fits(m, k, n)) return XTVXY_ERROR_UNSUPPORTED;
  // any of G, X and W may turn out to need its copy where aligned16 is 0: the largest of the plans
  thread_local PlanCache<size_t> cache;
  *bytes = cache.get(m, k, n, (type * 8 + act) * 2 + (aligned16 != 0), [&] { return most_backward_bytes(type, m, k, n, act, aligned16); });
  return XTVXY_SUCCESS;
}

xtvxy_status backward_impl(int type, int64_t m, int64_t k, int64_t n, const void* G, int64_t ldg, const void* X,
                           int64_t ldx, const void* W, int64_t ldw, const void* pre, int64_t ldp, int act, void* dX,
                           int64_t lddx, void* dW, int64_t lddw, float* db, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  if (m < 0 || k < 0 || n < 0 || !valid_act(act)) return XTVXY_ERROR_INVALID_VALUE;
  if (padded_overflow(m, n)) return XTVXY_ERROR_INVALID_VALUE;
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

  const BackwardPlan& p = plan_backward(type, m, k, n, act, whole_chunks(mg), whole_chunks(mx), whole_chunks(mw),
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
    take_plan(&a.dx, p.dx, base + p.dx_off);
    a.dx.e = {nullptr, nullptr, 0, nullptr, 0, dX, lddx, XTVXY_ACT_NONE};
  }
  if (dW && k > 0) {
    a.dw.B = X;
    a.dw.ldb = ldx;
    a.dw.m = n;
    a.dw.n = k;
    a.dw.k = m;
    take_plan(&a.dw, p.dw, base + p.dw_off);
    a.dw.e = {nullptr, nullptr, 0, nullptr, 0, dW, lddw, XTVXY_ACT_NONE};
  }
  a.dx.type = a.dw.type = type;
  a.dw_first = m > n;
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
