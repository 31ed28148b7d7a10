// Host side of the losses over an output layer's logits and their gradients: argument checks, the pieces of the
// vocabulary, the plans of the products, the workspace, and the launches. Argument errors are found before
// anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "linear_plan.h"
#include "loss.h"

using namespace xtvxy;

namespace {

// Most bytes of a piece's d, and of the statistics or copies of a piece's forward pass. Pieces of fewer classes
// than kLeastPiece would leave the products of the gradient without depth.
constexpr int64_t kPieceBytes = (int64_t)1 << 29;
constexpr int64_t kLeastPiece = 4096;
constexpr double kMemoryUs = 8.0;  // what logits in memory cost besides their product
constexpr int64_t kMostMemoryRows = 65535 * kMemoryRows;  // their second grid dimension
// The sum of dX's parts: a launch, and the parts read (4 slices of 67 MB and the result: 86 us).
constexpr double kFinishUs = 8.0, kPartsBytesPerUs = 3.5e6;
// What d costs more from memory than from the cache (8192 x 65536 of bf16: 300 us, 4096 x 100000 190).
constexpr double kCachedBytesPerUs = 4e6;

// Pieces of a vocabulary of n of at most `bytes` with `per_class` of them a class, all of one width but the last.
int64_t piece_of(int64_t n, int64_t per_class, int64_t most) {
  most = std::min(most, std::max<int64_t>(kLeastPiece, kPieceBytes / std::max<int64_t>(per_class, 1)) / 256 * 256);
  if (n <= most) return n;
  return cdiv(cdiv(n, cdiv(n, most)), 256) * 256;
}

// Classes of a piece up to which its launches fit.
int64_t most_classes(int64_t m, int64_t k, int es) {
  int64_t most = kRingMaxPitch / es;  // a row of d
  const int64_t tile_rows = cdiv(m, 64);
  if (tile_rows > 0) most = std::min(most, kMaxGroups / tile_rows * 64);
  return most / 256 * 256;
}

bool shape_fits(int64_t m, int64_t k, int64_t n, int es) {
  const int64_t most = most_classes(m, k, es);
  return k <= kRingMaxPitch / es && most >= kLeastPiece && n <= INT32_MAX && m <= INT32_MAX &&
         backward_fits(m, k, std::min(n, most));
}

// Workspace of the lists' order for tiles of this edge; nothing where the lists are searched.
struct OrderPlan {
  ListOrder order{};
  size_t starts = 0, bytes = 0;
};
OrderPlan plan_order(int64_t m, int64_t n, int64_t per_row, int tile) {
  OrderPlan p;
  p.order.half = tile / 2;
  p.order.columns = cdiv(n, p.order.half);
  p.order.strip_rows = strip_rows_of(tile);
  if (!order_pays(m, n, per_row) || p.order.columns > kMostHalves) return p;
  const int64_t strips = cdiv(m, p.order.strip_rows);
  p.starts = align_up((size_t)strips * (p.order.columns + 1) * 4);
  p.bytes = p.starts + align_up((size_t)strips * p.order.strip_rows * per_row * 4);
  return p;
}

// The order made, or none.
hipError_t order_lists(const OrderPlan& p, const ClassList& list, const float* weights, int64_t m, int64_t n, char* ws,
                       ListOrder* order, hipStream_t s) {
  *order = p.order;
  if (p.bytes == 0) return hipSuccess;
  order->starts = reinterpret_cast<uint32_t*>(ws);
  order->entries = reinterpret_cast<uint32_t*>(ws + p.starts);
  return launch_list_order({list, *order, weights, m, n}, s);
}

// Up to 64 rows of 16 bits over so many classes that reading W is what counts: tiles of 128 have more of it under way
// than those of 64. us: 64 x 1024 x 131072 67, 84; 33 x 3500 x 20000 89, 91; fp32, bound by the matrix unit, 129, 82.
int loss_tile(int type, int64_t m, int64_t n) { return type != kF32 && m <= 64 && n >= 128 * kComputeUnits / 2 ? 128 : 0; }

// Few tiles over a long contraction: their products are split over it, and the logits' parts joined in memory, where that
// pays in spite of the launches more. us, with their gradient: fp32 924 x 4072 x 144 184 to 87, 93 x 1415 x 105 77 to 49;
// bf16 500 x 4096 x 300 56 to 44.
struct MemoryPlan {
  ProductPlan product;
  size_t parts_off = 0, logits_off = 0;
  bool used = false;
};
MemoryPlan plan_memory(int type, int64_t m, int64_t k, int64_t n, const ProductPlan& tiles) {
  MemoryPlan p;
  if (n > kFewClasses || m > kMostMemoryRows || m * n * 4 > kPieceBytes / 4) return p;
  p.product = plan_product(type, m, n, k, true);
  // every tile split: whole ones would be stored by the product's own epilogue, in its element type
  p.used = p.product.splits > 1 && p.product.whole == 0 && p.product.us + kMemoryUs < tiles.us;
  return p;
}

struct ForwardPlan {
  bool pack_x, pack_w;
  int64_t piece;
  ProductPlan whole, last;  // of a piece, of the last one
  int64_t parts;            // halves of tiles' columns of a piece
  OrderPlan order;
  MemoryPlan memory;
  FewPlan few;              // of few rows: their products go through the workspace, whatever the operands' alignment
  size_t x_off, w_off, stats_off, run_off, listed_off, order_off, logits_off, bytes = 0;
};

ForwardPlan make_forward_plan(int type, int64_t m, int64_t k, int64_t n, int64_t per_row, bool x_whole, bool w_whole) {
  ForwardPlan p;
  const int es = elem_size(type);
  const auto take = [&](bool want, size_t bytes) {
    const size_t at = p.bytes;
    if (want) p.bytes += align_up(bytes);
    return at;
  };
  // Few rows: one pass over W that keeps more of it under way than tiles do, then a pass over their logits. us, against
  // tiles: bf16 1 x 4096 x 32000 53, 62; 1 x 2048 x 131072 94, 115; 7 x 512 x 100000 28, 34; fp32 16 x 4096 x 16000 63, 83;
  // but of 17 rows and more of 16 bits 32 x 512 x 50000 23, 19, 32 x 1024 x 131072 78, 73, unless rows need copies.
  if (m <= 16 || type == kF32 || !x_whole || !w_whole) p.few = plan_few(type, m, k, n);
  p.pack_x = p.pack_w = false;
  if (p.few.waves > 0) {
    const int64_t splits = p.few.product.splits;
    p.piece = piece_of(n, m * splits * 4, most_classes(m, k, es));
    p.stats_off = take(true, (size_t)cdiv(p.piece, kFewChunk) * m * 8);
    p.run_off = take(p.piece < n, (size_t)m * 8);
    p.listed_off = take(true, (size_t)m * per_row * 4);
    p.logits_off = take(true, (size_t)splits * m * p.piece * 4);
    return p;
  }
  p.pack_x = !x_whole;
  p.pack_w = !w_whole;
  // statistics: 8 bytes a row and half tile of at least 32 classes
  const int64_t per_class = std::max<int64_t>(m / 4, p.pack_w ? padded(k, es) * es : 0);
  p.piece = piece_of(n, per_class, most_classes(m, k, es));
  p.whole = plan_product(type, m, p.piece, k, true, false, loss_tile(type, m, p.piece));
  const int64_t last = n - (cdiv(n, std::max<int64_t>(p.piece, 1)) - 1) * p.piece;
  p.last = p.piece == n ? p.whole : plan_product(type, m, last, k, true, false, p.whole.tile);
  p.parts = 2 * cdiv(p.piece, p.whole.tile);
  if (p.piece == n) p.memory = plan_memory(type, m, k, n, p.whole);
  p.x_off = take(p.pack_x, packed_bytes(m, k, es));
  p.w_off = take(p.pack_w, packed_bytes(p.piece, k, es));
  p.stats_off = take(true, (size_t)p.parts * m * 8);
  p.run_off = take(p.piece < n, (size_t)m * 8);
  p.listed_off = take(true, (size_t)m * per_row * 4);
  if (!p.memory.used) p.order = plan_order(m, n, per_row, p.whole.tile);
  p.order_off = take(true, p.order.bytes);
  p.memory.parts_off = take(p.memory.used, p.memory.product.bytes);
  p.memory.logits_off = take(p.memory.used, (size_t)m * n * 4);
  return p;
}

const ForwardPlan& plan_forward(int type, int64_t m, int64_t k, int64_t n, int64_t per_row, bool x_whole, bool w_whole) {
  thread_local PlanCache<ForwardPlan> cache;
  return cache.get(m, k, n, ((per_row * 4 + type) * 2 + x_whole) * 2 + w_whole,
                   [&] { return make_forward_plan(type, m, k, n, per_row, x_whole, w_whole); });
}

struct BackwardPlan {
  bool pack_x, pack_w, parts;
  int64_t piece, pieces, ldd;
  int64_t slice = 0, slices = 0;  // floats of a part of dX, parts that there is room for
  ProductPlan logits, last_logits, dx, dw, last_dx, last_dw;
  OrderPlan order;
  MemoryPlan memory;
  size_t x_off, w_off, d_off, factor_off, scale_off, sums_off, dx_off, dw_off, order_off, bytes = 0;
};

// The products of pieces of that many classes.
void plan_pieces(BackwardPlan* p, int type, int64_t m, int64_t k, int64_t n, int64_t piece, bool want_dx, bool want_dw) {
  p->piece = piece;
  p->pieces = cdiv(n, piece);
  p->parts = p->pieces > 1;
  p->ldd = cdiv(piece, 8) * 8;
  const int64_t last = n - (p->pieces - 1) * piece;
  p->logits = plan_product(type, m, piece, k, true, false, loss_tile(type, m, piece));
  p->last_logits = p->parts ? plan_product(type, m, last, k, true, false, p->logits.tile) : p->logits;
  plan_gradient(type, m, k, piece, want_dx, want_dw, true, &p->dx, &p->dw, 0, p->parts);
  p->last_dx = p->dx;
  p->last_dw = p->dw;
  const int tile = want_dx ? p->dx.tile : p->dw.tile;
  if (p->parts && (want_dx || want_dw)) plan_gradient(type, m, k, last, want_dx, want_dw, true, &p->last_dx, &p->last_dw, tile, true);
}

BackwardPlan make_backward_plan(int type, int64_t m, int64_t k, int64_t n, int64_t per_row, bool x_whole, bool w_whole, bool want_dx, bool want_dw) {
  BackwardPlan p;
  const int es = elem_size(type);
  want_dx = want_dx && k > 0;
  want_dw = want_dw && k > 0;
  p.pack_x = !x_whole;
  p.pack_w = !w_whole;
  // Of the numbers of pieces that fit, the one with the least estimated time: small ones stay in the cache, and their tiles
  // may leave CUs without work. (In pieces of up to 128, 256, 512 MiB and 1 GiB, ms with the forward pass: bf16 8192 x
  // 2048 x 65536 6.65, 6.85, 6.81, 6.83; 4096 x 128 x 100000 1.08, 1.13, 1.23, 1.24; 4096 x 1023 x 30000 1.22, 1.10, 1.12,
  // 1.13; fp32 4096 x 512 x 50000 6.73, 6.76, 6.24, 6.29.)
  const int64_t per_class = m * es + (p.pack_w ? padded(k, es) * es : 0), most = most_classes(m, k, es);
  const int64_t fewest = cdiv(n, piece_of(n, per_class, most));
  double least = 0;
  for (int64_t pieces : {fewest, fewest + 1, fewest + 2, fewest + 3, 2 * fewest, 2 * fewest + 1, 3 * fewest, 4 * fewest,
                         5 * fewest, 8 * fewest}) {
    const int64_t piece = pieces == 1 ? n : cdiv(cdiv(n, pieces), 256) * 256;
    if (pieces > fewest && piece < kLeastPiece) continue;
    BackwardPlan q = p;
    plan_pieces(&q, type, m, k, n, piece, want_dx, want_dw);
    const double slices = q.parts && want_dx ? (q.pieces - 1) * q.dx.splits + q.last_dx.splits : 0;
    // d of more than 128 MiB leaves the cache between its kernel and the products
    const double size = (double)m * piece * es, out = std::min(1.0, std::max(0.0, size / ((int64_t)1 << 27) - 1.0));
    const double us = out * m * n * es / kCachedBytesPerUs + (q.pieces - 1) * (q.logits.us + q.dx.us) + q.last_logits.us + q.last_dx.us + 6.0 * q.pieces +
                      (slices > 0 ? kFinishUs + slices * m * k * 4 / kPartsBytesPerUs : 0.0);
    if (least == 0 || us < least) {
      least = us;
      p = q;
    }
  }
  const int tile = want_dx ? p.dx.tile : p.dw.tile;
  size_t dx_bytes = p.dx.bytes;
  if (p.parts && want_dx) {  // dX's sums over the pieces join in the end, or whenever they fill their place
    p.dx.whole = p.last_dx.whole = 0;
    p.slice = cdiv(m, tile) * cdiv(k, tile) * tile * tile;
    const int64_t all = (p.pieces - 1) * p.dx.splits + p.last_dx.splits, more = std::max(p.dx.splits, p.last_dx.splits);
    p.slices = std::min(all, std::max(more + 1, kPieceBytes / (p.slice * 4)));
    dx_bytes = (size_t)p.slices * p.slice * 4;
  }
  const auto take = [&](bool want, size_t bytes) {
    const size_t at = p.bytes;
    if (want) p.bytes += align_up(bytes);
    return at;
  };
  p.x_off = take(p.pack_x, packed_bytes(m, k, es));
  p.w_off = take(p.pack_w, packed_bytes(p.piece, k, es));
  p.d_off = take(want_dx || want_dw, (size_t)m * p.ldd * es);
  p.factor_off = take(true, (size_t)m * 4);
  p.scale_off = take(type != kF32, 8);
  if (!p.parts) p.memory = plan_memory(type, m, k, n, p.logits);
  const int64_t rows = p.memory.used ? cdiv(m, kMemoryRows) : cdiv(m, p.logits.tile) * 2;
  p.sums_off = take(true, (size_t)rows * p.piece * 4);
  p.dx_off = take(want_dx, dx_bytes);
  p.dw_off = take(want_dw, std::max(p.dw.bytes, p.last_dw.bytes));
  if (!p.memory.used) p.order = plan_order(m, n, per_row, p.logits.tile);
  p.order_off = take(true, p.order.bytes);
  p.memory.parts_off = take(p.memory.used, p.memory.product.bytes);
  p.memory.logits_off = take(p.memory.used, (size_t)m * n * 4);
  return p;
}

const BackwardPlan& plan_backward(int type, int64_t m, int64_t k, int64_t n, int64_t per_row, bool x_whole, bool w_whole, bool want_dx, bool want_dw) {
  thread_local PlanCache<BackwardPlan> cache;
  return cache.get(m, k, n, ((((per_row * 4 + type) * 2 + x_whole) * 2 + w_whole) * 2 + want_dx) * 2 + want_dw,
                   [&] { return make_backward_plan(type, m, k, n, per_row, x_whole, w_whole, want_dx, want_dw); });
}

xtvxy_status check_shape(int64_t m, int64_t k, int64_t n, int64_t per_row, int es) {
  if (m < 0 || k < 0 || n < 0 || per_row < 0) return XTVXY_ERROR_INVALID_VALUE;
  if (padded_overflow(m, n) || padded_overflow(m, k) || padded_overflow(n, k) || bytes_overflow(m, per_row))
    return XTVXY_ERROR_INVALID_VALUE;
  if (per_row > kMostListed || !shape_fits(m, k, n, es)) return XTVXY_ERROR_UNSUPPORTED;
  return XTVXY_SUCCESS;
}

// The largest of the plans that the operands' alignment may lead to.
template <typename Fn>
size_t most_bytes(int64_t k, int es, int aligned16, Fn bytes) {
  const bool chunks = k * es % 16 == 0;
  size_t most = 0;
  for (int x = 0; x < 2; ++x)
    for (int w = 0; w < 2; ++w)
      if (!aligned16 || !chunks || (x && w)) most = std::max(most, bytes(chunks && x, chunks && w));
  return most;
}

xtvxy_status forward_workspace(int type, int64_t m, int64_t k, int64_t n, int64_t per_row, int aligned16, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  const xtvxy_status st = check_shape(m, k, n, per_row, elem_size(type));
  if (st != XTVXY_SUCCESS) return st;
  *bytes = m == 0 || n == 0 ? 0 : most_bytes(k, elem_size(type), aligned16, [&](bool x, bool w) {
    return plan_forward(type, m, k, n, per_row, x, w).bytes;
  });
  return XTVXY_SUCCESS;
}

xtvxy_status backward_workspace(int type, int64_t m, int64_t k, int64_t n, int64_t per_row, int aligned16, size_t* bytes) {
  if (!bytes) return XTVXY_ERROR_NULL_POINTER;
  const xtvxy_status st = check_shape(m, k, n, per_row, elem_size(type));
  if (st != XTVXY_SUCCESS) return st;
  *bytes = m == 0 || n == 0 ? 0 : most_bytes(k, elem_size(type), aligned16, [&](bool x, bool w) {
    size_t most = 0;  // a product alone may be split further than the two together
    for (int want = 0; want < 4; ++want)
      most = std::max(most, plan_backward(type, m, k, n, per_row, x, w, want & 1, want & 2).bytes);
    return most;
  });
  return XTVXY_SUCCESS;
}

bool bad_workspace(size_t need, const void* ws, size_t bytes) {
  return need > 0 && (!ws || bytes < need || reinterpret_cast<uintptr_t>(ws) % kAlign != 0);
}

Matrix list_of(const ClassList& l, int64_t m) { return {l.p, m, l.per_row, std::max<int64_t>(l.ld, 1), l.bits / 8}; }

bool any_overlap(const Matrix* written, int outputs, const Matrix* read, int inputs) {
  for (int o = 0; o < outputs; ++o) {
    for (int i = 0; i < inputs; ++i)
      if (overlap(written[o], read[i])) return true;
    for (int q = 0; q < o; ++q)
      if (overlap(written[o], written[q])) return true;
  }
  return false;
}

struct Layer {
  int type;
  int64_t m, k, n;
  const void* X;
  int64_t ldx;
  const void* W;
  int64_t ldw;
  const float* bias;
  int es() const { return elem_size(type); }
  Matrix mx() const { return {X, m, k, ldx, es()}; }
  Matrix mw() const { return {W, n, k, ldw, es()}; }
  bool bad() const { return bad_ld(ldx, k, m) || bad_ld(ldw, k, n); }
  bool missing() const { return m > 0 && n > 0 && k > 0 && (!X || !W); }
  const void* rows_of_w(const void* w, int64_t ld, int64_t j) const { return static_cast<const char*>(w) + j * ld * es(); }
};

// X's and a piece of W's copies where their rows do not suit the products, which `a` takes then.
hipError_t pack_operands(const Layer& l, bool pack_x, bool pack_w, void* x_copy, void* w_copy, int64_t j, int64_t classes,
                         ProductArgs* a, hipStream_t s) {
  const int es = l.es();
  const int64_t ld = padded(l.k, es);
  PackArgs pack{};
  a->A = l.X;
  a->lda = l.ldx;
  a->B = l.rows_of_w(l.W, l.ldw, j);
  a->ldb = l.ldw;
  if (pack_x) {
    if (j == 0) pack.job[pack.jobs++] = {l.X, x_copy, l.ldx, ld, l.m, l.k};
    a->A = x_copy;
    a->lda = ld;
  }
  if (pack_w) {
    pack.job[pack.jobs++] = {a->B, w_copy, l.ldw, ld, classes, l.k};
    a->B = w_copy;
    a->ldb = ld;
  }
  a->m = l.m;
  a->n = classes;
  a->k = l.k;
  a->type = l.type;
  return pack.jobs > 0 && l.k > 0 ? launch_pack(pack, l.type, s) : hipSuccess;
}

// The logits of one piece as fp32 in memory, which `a` has as its one part then.
hipError_t logits_in_memory(ProductArgs* a, const MemoryPlan& p, char* base, hipStream_t s) {
  take_plan(a, p.product, base + p.parts_off);
  hipError_t e = launch_layer_ring(*a, s);
  if (e != hipSuccess) return e;
  float* logits = reinterpret_cast<float*>(base + p.logits_off);
  ProductArgs sum = *a;
  sum.type = kF32;  // of what is written; the parts are fp32 in any case
  sum.e = {nullptr, nullptr, 0, nullptr, 0, logits, a->n, XTVXY_ACT_NONE};
  e = launch_product_finish(sum, s);
  a->partial = logits;
  a->splits = 1;
  return e;
}

// A teacher's logits; labels: teacher null.
struct Teacher {
  const void* logits;
  int64_t ld;
  int32_t type;
  float temperature;
  float* weights;
};

bool valid_temperature(float t) { return t > 0.0f && std::isfinite(t) && std::isfinite(1.0f / t); }

xtvxy_status forward_impl(const Layer& l, const ClassList& list, const Teacher* teacher, float* loss, float* lse, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
  const int es = l.es();
  const xtvxy_status st = check_shape(l.m, l.k, l.n, list.per_row, es);
  if (st != XTVXY_SUCCESS) return st;
  if (l.bad() || (list.bits != 32 && list.bits != 64) || bad_ld(list.ld, list.per_row, l.m)) return XTVXY_ERROR_INVALID_VALUE;
  const int64_t m = l.m, n = l.n;
  if (m == 0) return XTVXY_SUCCESS;
  if (!loss || !lse || l.missing() || (list.per_row > 0 && !list.p)) return XTVXY_ERROR_NULL_POINTER;
  if (teacher && list.per_row > 0 && (!teacher->logits || !teacher->weights)) return XTVXY_ERROR_NULL_POINTER;
  Matrix read[] = {l.mx(), l.mw(), vec(l.bias, n), list_of(list, m), {}};
  Matrix written[] = {vec(loss, m), vec(lse, m), {}};
  if (teacher) {
    read[4] = {teacher->logits, m, list.per_row, teacher->ld, teacher->type == XTVXY_TYPE_F32 ? 4 : 2};
    written[2] = vec(teacher->weights, m * list.per_row);
  }
  if (any_overlap(written, 3, read, 5)) return XTVXY_ERROR_ALIASING;
  const float inv_temperature = teacher ? 1.0f / teacher->temperature : 1.0f;
  // without classes: the logarithm of an empty sum, and every label is beyond the vocabulary
  const ForwardPlan p = n > 0 ? plan_forward(l.type, m, l.k, n, list.per_row, whole_chunks(l.mx()), whole_chunks(l.mw())) : ForwardPlan{};
  if (bad_workspace(p.bytes, ws, ws_bytes)) return XTVXY_ERROR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  float* weights = teacher ? teacher->weights : nullptr;
  TeacherArgs t{};
  if (teacher && list.per_row > 0) {
    const int type = teacher->type == XTVXY_TYPE_F32 ? kF32 : teacher->type == XTVXY_TYPE_BF16 ? kBf16 : kF16;
    t = {list, teacher->logits, teacher->ld, type, inv_temperature, m, n, weights};
    if (list.per_row > kLaneListed) {
      if (launch_teacher_weights(t, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
      t.teacher = nullptr;
    }
  }
  float* stats = reinterpret_cast<float*>(base + p.stats_off);
  LossFinishArgs f{stats, 0, m, n, p.piece < n ? reinterpret_cast<float*>(base + p.run_off) : nullptr, 1, n == 0, list,
                   reinterpret_cast<float*>(base + p.listed_off), weights, loss, lse, t};
  if (teacher && list.per_row == 0) f.weights = loss;  // no terms: never read
  if (n == 0) return status_of(launch_loss_finish(f, stream));
  ListOrder order;
  if (order_lists(p.order, list, t.teacher ? nullptr : weights, m, n, base + p.order_off, &order, stream) != hipSuccess)
    return XTVXY_ERROR_LAUNCH;
  for (int64_t j = 0; j < n; j += p.piece) {
    const int64_t classes = std::min(p.piece, n - j);
    LossForwardArgs a{};
    if (pack_operands(l, p.pack_x, p.pack_w, base + p.x_off, base + p.w_off, j, classes, &a.product, stream) != hipSuccess)
      return XTVXY_ERROR_LAUNCH;
    f.first = j == 0;
    f.last = j + classes == n;
    take_plan(&a.product, f.last ? p.last : p.whole, nullptr);
    if (p.few.waves > 0) {
      take_plan(&a.product, p.few.product, base + p.logits_off);
      a.product.in_parts = 1;
      if (launch_product_few(a.product, p.few.waves, p.few.outputs, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    }
    if (p.memory.used && logits_in_memory(&a.product, p.memory, base, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    a.bias = l.bias ? l.bias + j : nullptr;
    a.inv_temperature = inv_temperature;
    a.first_class = j;
    a.list = list;
    a.order = order;
    a.listed = reinterpret_cast<float*>(base + p.listed_off);
    a.stats = stats;
    if (p.memory.used || (p.few.waves > 0 && f.first && f.last && n <= kFewClasses)) return status_of(launch_loss_few_rows(a, f, stream));
    if ((p.few.waves > 0 ? launch_loss_few(a, stream) : launch_loss_forward(a, stream)) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    f.parts = p.few.waves > 0 ? cdiv(classes, kFewChunk) : 2 * cdiv(classes, a.product.tile);
    if (launch_loss_finish(f, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  return XTVXY_SUCCESS;
}

struct Gradients {
  void* dX;
  int64_t lddx;
  void* dW;
  int64_t lddw;
  float* db;
};

xtvxy_status backward_impl(const Layer& l, const float* grad, const ClassList& list, const float* weights, bool labels,
                           float temperature, const float* lse, const Gradients& o, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  const int es = l.es();
  const xtvxy_status st = check_shape(l.m, l.k, l.n, list.per_row, es);
  if (st != XTVXY_SUCCESS) return st;
  const int64_t m = l.m, k = l.k, n = l.n;
  if (l.bad() || (list.bits != 32 && list.bits != 64) || bad_ld(list.ld, list.per_row, m) || (o.dX && bad_ld(o.lddx, k, m)) ||
      (o.dW && bad_ld(o.lddw, k, n)))
    return XTVXY_ERROR_INVALID_VALUE;
  const bool want = o.dX || o.dW || o.db, reads = m > 0 && n > 0 && want;
  if (reads && (!grad || !lse || l.missing() || (list.per_row > 0 && (!list.p || (!labels && !weights))))) return XTVXY_ERROR_NULL_POINTER;
  const Matrix read[] = {l.mx(), l.mw(), vec(l.bias, n), list_of(list, m), vec(grad, m), vec(lse, m), vec(weights, m * list.per_row)};
  const Matrix written[] = {{o.dX, m, k, o.lddx, es}, {o.dW, n, k, o.lddw, es}, vec(o.db, n)};
  if (any_overlap(written, 3, read, 7)) return XTVXY_ERROR_ALIASING;
  GradientArgs g{};
  g.dx.type = g.dw.type = l.type;
  g.dx.m = o.dX && k > 0 ? m : 0;
  g.dw.m = o.dW && k > 0 ? n : 0;
  g.dx.n = g.dw.n = k;
  g.dx.e = {nullptr, nullptr, 0, nullptr, 0, o.dX, o.lddx, XTVXY_ACT_NONE};
  g.dw.e = {nullptr, nullptr, 0, nullptr, 0, o.dW, o.lddw, XTVXY_ACT_NONE};
  if (!reads) {  // the products' empty sums
    if (!want) return XTVXY_SUCCESS;
    if (o.db && n > 0 && launch_zero(o.db, (size_t)n * 4, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    ProductPlan none;
    none.k_per_split = kTileDepth;
    take_plan(&g.dx, none, nullptr);
    take_plan(&g.dw, none, nullptr);
    return status_of(launch_gradient_tile(g, l.type, stream));
  }
  const BackwardPlan& p = plan_backward(l.type, m, k, n, list.per_row, whole_chunks(l.mx()), whole_chunks(l.mw()), g.dx.m > 0, g.dw.m > 0);
  if (bad_workspace(p.bytes, ws, ws_bytes)) return XTVXY_ERROR_WORKSPACE;
  char* base = static_cast<char*>(ws);
  float* factor = reinterpret_cast<float*>(base + p.factor_off);
  float* scale = l.type == kF16 || (l.type == kBf16 && labels) ? reinterpret_cast<float*>(base + p.scale_off) : nullptr;
  const float inv_temperature = 1.0f / temperature;
  const float* target = labels ? nullptr : list.per_row > 0 ? weights : factor;  // none listed: never read
  if (launch_loss_factor({grad, list, target, inv_temperature, m, n, factor, scale}, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  ListOrder order;
  if (order_lists(p.order, list, target, m, n, base + p.order_off, &order, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  const bool products = g.dx.m > 0 || g.dw.m > 0;
  int64_t slices = 0;  // of dX's sums so far
  for (int64_t j = 0; j < n; j += p.piece) {
    const int64_t classes = std::min(p.piece, n - j);
    const bool last = j + classes == n;
    LossGradientArgs a{};
    if (pack_operands(l, p.pack_x, p.pack_w, base + p.x_off, base + p.w_off, j, classes, &a.product, stream) != hipSuccess)
      return XTVXY_ERROR_LAUNCH;
    take_plan(&a.product, last ? p.last_logits : p.logits, nullptr);
    a.bias = l.bias ? l.bias + j : nullptr;
    a.inv_temperature = inv_temperature;
    a.first_class = j;
    a.list = list;
    a.order = order;
    a.weights = target;
    a.factor = factor;
    a.lse = lse;
    a.scale = scale;
    a.d = products ? base + p.d_off : nullptr;
    a.ldd = cdiv(classes, 8) * 8;
    a.sums = o.db ? reinterpret_cast<float*>(base + p.sums_off) : nullptr;
    int64_t sum_rows = 2 * cdiv(m, a.product.tile);
    if (p.memory.used) {
      if (logits_in_memory(&a.product, p.memory, base, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
      if (launch_loss_gradient_memory(a, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
      sum_rows = cdiv(m, kMemoryRows);
    } else if (launch_loss_gradient(a, stream) != hipSuccess) {
      return XTVXY_ERROR_LAUNCH;
    }

    GradientArgs piece = g;
    const ProductPlan &dx = last ? p.last_dx : p.dx, &dw = last ? p.last_dw : p.dw;
    piece.dx.A = piece.dw.A = a.d;
    piece.dx.lda = piece.dw.lda = a.ldd;
    piece.dx.B = a.product.B;
    piece.dx.ldb = a.product.ldb;
    piece.dw.B = a.product.A;
    piece.dw.ldb = a.product.lda;
    piece.dx.k = classes;
    piece.dw.k = m;
    piece.dw.m = g.dw.m > 0 ? classes : 0;
    piece.dw.e.out = o.dW ? static_cast<char*>(o.dW) + j * o.lddw * es : nullptr;
    piece.dx.scale = piece.dw.scale = scale ? scale + 1 : nullptr;
    take_plan(&piece.dx, dx, base + p.dx_off);
    take_plan(&piece.dw, dw, base + p.dw_off);
    const int tile = g.dx.m > 0 ? dx.tile : dw.tile;
    if (p.parts && g.dx.m > 0) {
      if (slices + dx.splits > p.slices) {
        if (launch_sum_slices(reinterpret_cast<float*>(base + p.dx_off), slices, p.slice, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
        slices = 1;
      }
      piece.dx.in_parts = 1;
      piece.dx.whole = 0;
      piece.dx.partial += slices * p.slice;
      slices += dx.splits;
    }
    piece.dw_first = m > classes;
    piece.n = classes;
    piece.db = o.db ? o.db + j : nullptr;
    piece.sums = a.sums;
    piece.sum_rows = sum_rows;
    if (launch_gradient_ring(piece, l.type, tile, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    piece.db = nullptr;
    if (p.parts && g.dx.m > 0) {  // all pieces' parts at once, after the last
      piece.dx.partial = reinterpret_cast<float*>(base + p.dx_off);
      piece.dx.splits = (int32_t)slices;
      if (!last) piece.dx.m = 0;
    }
    if (launch_gradient_finish(piece, l.type, stream) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  }
  return XTVXY_SUCCESS;
}

ClassList labels_of(const void* labels, int bits) { return {labels, 1, bits, 1}; }

bool valid_list(int64_t per_row) { return per_row >= 0 && per_row <= INT32_MAX; }
bool valid_type(int t) { return t == XTVXY_TYPE_F32 || t == XTVXY_TYPE_BF16 || t == XTVXY_TYPE_F16; }

xtvxy_status distillation(const Layer& l, int64_t s, const void* classes, int64_t ldc, int bits, const void* teacher,
                          int64_t ldt, int teacher_type, float temperature, float* loss, float* lse, float* weights,
                          void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!valid_list(s) || !valid_type(teacher_type) || !valid_temperature(temperature) || l.m < 0 || bad_ld(ldt, s, l.m))
    return XTVXY_ERROR_INVALID_VALUE;
  const Teacher t{teacher, ldt, teacher_type, temperature, weights};
  return forward_impl(l, {classes, ldc, bits, (int32_t)s}, &t, loss, lse, ws, ws_bytes, stream);
}

xtvxy_status distillation_backward(const Layer& l, int64_t s, const float* grad, const void* classes, int64_t ldc, int bits,
                                   const float* weights, float temperature, const float* lse, const Gradients& o, void* ws,
                                   size_t ws_bytes, hipStream_t stream) {
  if (!valid_list(s) || !valid_temperature(temperature)) return XTVXY_ERROR_INVALID_VALUE;
  return backward_impl(l, grad, {classes, ldc, bits, (int32_t)s}, weights, false, temperature, lse, o, ws, ws_bytes, stream);
}

}  // namespace

extern "C" {

#define XTVXY_LOSS(SUFFIX, TYPE, T)                                                                                     \
  xtvxy_status xtvxy_linear_cross_entropy_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n, int aligned16,     \
                                                                    size_t* bytes) {                                    \
    return forward_workspace(TYPE, m, k, n, 1, aligned16, bytes);                                                       \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_cross_entropy_##SUFFIX(int64_t m, int64_t k, int64_t n, const T* X, int64_t ldx, const T* W,  \
                                                   int64_t ldw, const float* bias, const void* labels,                  \
                                                   int index_bits, float* loss, float* lse, void* workspace,            \
                                                   size_t workspace_bytes, hipStream_t stream) {                        \
    return forward_impl({TYPE, m, k, n, X, ldx, W, ldw, bias}, labels_of(labels, index_bits), nullptr, loss, lse,       \
                        workspace, workspace_bytes, stream);                                                            \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_cross_entropy_backward_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n,           \
                                                                             int aligned16, size_t* bytes) {            \
    return backward_workspace(TYPE, m, k, n, 1, aligned16, bytes);                                                      \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_cross_entropy_backward_##SUFFIX(                                                            \
      int64_t m, int64_t k, int64_t n, const float* grad, const T* X, int64_t ldx, const T* W, int64_t ldw,             \
      const float* bias, const void* labels, int index_bits, const float* lse, T* dX, int64_t lddx, T* dW,              \
      int64_t lddw, float* db, void* workspace, size_t workspace_bytes, hipStream_t stream) {                           \
    return backward_impl({TYPE, m, k, n, X, ldx, W, ldw, bias}, grad, labels_of(labels, index_bits), nullptr, true,     \
                         1.0f, lse, {dX, lddx, dW, lddw, db}, workspace, workspace_bytes, stream);                      \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_distillation_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n, int64_t s,          \
                                                                   int aligned16, size_t* bytes) {                      \
    return forward_workspace(TYPE, m, k, n, s, aligned16, bytes);                                                       \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_distillation_##SUFFIX(                                                                      \
      int64_t m, int64_t k, int64_t n, const T* X, int64_t ldx, const T* W, int64_t ldw, const float* bias, int64_t s,  \
      const void* classes, int64_t ldc, int index_bits, const void* teacher, int64_t ldt, int teacher_type,             \
      float temperature, float* loss, float* lse, float* weights, void* workspace, size_t workspace_bytes,              \
      hipStream_t stream) {                                                                                             \
    return distillation({TYPE, m, k, n, X, ldx, W, ldw, bias}, s, classes, ldc, index_bits, teacher, ldt,               \
                        teacher_type, temperature, loss, lse, weights, workspace, workspace_bytes, stream);             \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_distillation_backward_##SUFFIX##_workspace_size(int64_t m, int64_t k, int64_t n, int64_t s, \
                                                                            int aligned16, size_t* bytes) {             \
    return backward_workspace(TYPE, m, k, n, s, aligned16, bytes);                                                      \
  }                                                                                                                     \
  xtvxy_status xtvxy_linear_distillation_backward_##SUFFIX(                                                             \
      int64_t m, int64_t k, int64_t n, const float* grad, const T* X, int64_t ldx, const T* W, int64_t ldw,             \
      const float* bias, int64_t s, const void* classes, int64_t ldc, int index_bits, const float* weights,             \
      float temperature, const float* lse, T* dX, int64_t lddx, T* dW, int64_t lddw, float* db, void* workspace,        \
      size_t workspace_bytes, hipStream_t stream) {                                                                     \
    return distillation_backward({TYPE, m, k, n, X, ldx, W, ldw, bias}, s, grad, classes, ldc, index_bits, weights,     \
                                 temperature, lse, {dX, lddx, dW, lddw, db}, workspace, workspace_bytes, stream);       \
  }

XTVXY_LOSS(f32, kF32, float)
XTVXY_LOSS(bf16, kBf16, uint16_t)
XTVXY_LOSS(f16, kF16, uint16_t)

}  // extern "C"
