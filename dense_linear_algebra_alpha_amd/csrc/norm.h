// Internal declarations of layer norm and its gradient (norm.cpp, norm.hip).
#pragma once

#include "linear.h"

namespace xtvxy {

struct NormArgs {
  const void* x;
  int64_t ldx;
  const float* weight;  // null: ones
  const float* bias;    // null: zeros
  void* out;
  int64_t ldo;
  float* mean;          // null: not wanted
  float* rstd;
  int64_t m, n;
  float eps;
};
hipError_t launch_norm(const NormArgs& a, int type, hipStream_t s);

struct NormGradientArgs {
  const void* g;
  const void* x;
  const float* mean;
  const float* rstd;
  const float* weight;  // null: ones
  void* dx;             // null: not wanted
  int64_t ldg, ldx, lddx;
  int64_t m, n;
  float* sums;          // [groups][2][n]: sums of g xhat and of g over the rows of a workgroup; null: not wanted
  int64_t groups;
  float* dweight;       // null: not wanted
  float* dbias;
};
// Workgroups of the gradient, each of which has column sums of its own.
int64_t norm_gradient_groups(int64_t m, int64_t n, int type);
constexpr int64_t kNormGradientMost = 16384;  // columns up to which a row stays in registers
hipError_t launch_norm_gradient(const NormGradientArgs& a, int type, hipStream_t s);

}  // namespace xtvxy
