// Internal declarations of the losses over an output layer's logits: softmax cross entropy and distillation from a
// teacher's top logits (loss.cpp, loss.hip).
#pragma once

#include "linear.h"

namespace xtvxy {

// Classes of each row that a loss looks at: labels (one a row) or a teacher's (per_row of them).
struct ClassList {
  const void* p;
  int64_t ld;
  int32_t bits, per_row;
};

// The lists' entries in the order in which the tiles look for them: of each strip of rows (those that a wavefront
// stages at a time) and each half tile of columns of the whole vocabulary, entries[starts[..]] up to the next start.
// An entry: row of the strip, column of the half tile, place in the list.
struct ListOrder {
  uint32_t* starts;      // [strips][columns + 1], null: the lists are searched
  uint32_t* entries;     // [strips][strip_rows * per_row]
  int64_t columns;       // half tiles
  int32_t strip_rows, half;  // half: classes of a half tile
};
// Half tiles up to which a workgroup counts them in LDS.
constexpr int64_t kMostHalves = 8192;
// The order is a launch of 3 to 6 us; searched lists cost every tile its rows' places. us, ordered and searched, with the
// gradient, bf16: 64 x 512 x 192 with 48 a row 45, 42; 512 x 512 x 4000 with 24 56, 48, with 48 60, 57; 1024 x 512 x 8000
// with 24 89, 87, with 48 93, 101; 4096 x 512 x 2000 with 24 91, 91, with 48 96, 104; 4096 x 512 x 16000 with 12 334, 351.
// Of these the rule misses one: it orders 512 x 512 x 4000 with 48.
inline bool order_pays(int64_t m, int64_t n, int64_t per_row) {
  return per_row >= 9 && (double)per_row * (1.0 + (double)m * n / (1 << 23)) >= 52.0;
}
inline int strip_rows_of(int tile) { return tile / 2 < 64 ? tile / 2 : 64; }
struct OrderArgs {
  ClassList list;
  ListOrder order;
  const float* weights;  // entries of weight zero are left out, null: none are
  int64_t m, n;
};
hipError_t launch_list_order(const OrderArgs& a, hipStream_t s);

// A piece of the logits t = (X W^T + bias) / T of which only statistics are kept: product.A is X, product.B the
// piece's rows of W, product.n its classes from `first_class` on.
struct LossForwardArgs {
  ProductArgs product;
  const float* bias;     // of the piece; null: zeros
  float inv_temperature;
  int64_t first_class;
  ClassList list;
  ListOrder order;
  float* listed;         // [m][per_row]: t of the listed classes of this piece
  float* stats;          // [2 tiles of columns][m][2]: largest t and sum of exp(t - largest) over half a tile
};
hipError_t launch_loss_forward(const LossForwardArgs& a, hipStream_t s);

// The same from a piece's products, of few rows, in memory: logits [splits][m][n], the parts to be added. Statistics of
// each kFewChunk classes, [chunks][m][2].
constexpr int64_t kFewChunk = 4096;
hipError_t launch_loss_few(const LossForwardArgs& a, hipStream_t s);

// Target weights from a teacher's logits: softmax(teacher / T) over a row's classes, equal classes' in the first.
constexpr int64_t kMostListed = 1024;
// Up to so many a row the launch that forms the loss forms the weights as well, a lane a class (a launch of 4 to 6 us less).
constexpr int64_t kLaneListed = 64;
struct TeacherArgs {
  ClassList list;
  const void* teacher;
  int64_t ldt;
  int32_t type;
  float inv_temperature;
  int64_t m, n;
  float* weights;
};
// Joins a piece's statistics into each row's running ones and, after the last piece, forms lse and loss.
struct LossFinishArgs {
  const float* stats;
  int64_t parts, m, n;
  float* run;            // [m][2], null: one piece
  int32_t first, last;
  ClassList list;
  const float* listed;
  const float* weights;  // [m][per_row], null: labels
  float* loss;
  float* lse;
  TeacherArgs teacher;   // teacher.teacher: the weights are formed first, null: they are there
};
hipError_t launch_loss_finish(const LossFinishArgs& a, hipStream_t s);

// Few rows' lse and loss from their logits in one launch: a workgroup a row, up to kFewClasses classes.
constexpr int64_t kFewClasses = 32768;
hipError_t launch_loss_few_rows(const LossForwardArgs& a, const LossFinishArgs& f, hipStream_t s);

// d from a product's logits in memory (product.partial: [m][n], one part), as launch_loss_gradient's; column sums of every
// kMemoryRows rows.
constexpr int64_t kMemoryRows = 8;
struct LossGradientArgs;
hipError_t launch_loss_gradient_memory(const LossGradientArgs& a, hipStream_t s);

// The weights in a launch of their own.
hipError_t launch_teacher_weights(const TeacherArgs& a, hipStream_t s);

// factor_i of d_ij = factor_i (softmax_ij - target_ij): grad_i / T, 0 for rows that do not count, NaN for bad ones; and
// scale[0] and scale[1] = 1 / scale[0] with which the largest |factor| becomes 2^13. For fp16 that keeps d in its range. For
// 16 bits and labels it takes a rounding away: most of d is its label's place, factor_i (softmax - 1), and under a mean all
// rows have one factor, whose rounding would be in all of them (bf16 566 x 384 x 7650, in the 2-norm: dX off
// by 2.46e-3, scaled 1.68e-3, of which its own rounding 1.65e-3); scaled that place is a power of two but for its softmax.
struct LossFactorArgs {
  const float* grad;
  ClassList list;
  const float* weights;  // null: labels
  float inv_temperature;
  int64_t m, n;
  float* factor;
  float* scale;          // null: not wanted
};
hipError_t launch_loss_factor(const LossFactorArgs& a, hipStream_t s);

// d of a piece, rounded to the product's type (times scale[0]) in rows of ldd elements, zero beyond the piece; and
// the column sums of each half tile of rows, unrounded and not scaled.
struct LossGradientArgs {
  ProductArgs product;
  const float* bias;
  float inv_temperature;
  int64_t first_class;
  ClassList list;
  ListOrder order;
  const float* weights;
  const float* factor;
  const float* lse;
  const float* scale;    // null: 1
  void* d;               // null: not wanted
  int64_t ldd;
  float* sums;           // [2 tiles of rows][n], null: not wanted
};
hipError_t launch_loss_gradient(const LossGradientArgs& a, hipStream_t s);

// slices[0] = the sum of `count` slices of `elements` floats (a multiple of 4) in their order.
hipError_t launch_sum_slices(float* slices, int64_t count, int64_t elements, hipStream_t s);

}  // namespace xtvxy
