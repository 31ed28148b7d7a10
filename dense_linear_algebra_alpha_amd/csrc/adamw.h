// Internal declarations of the AdamW step (adamw.cpp, adamw.hip).
#pragma once

#include "linear.h"

namespace xtvxy {

constexpr int kAdamBlock = 128;    // elements that share an exponent in 8-bit states
constexpr int kAdamChunk = 2048;   // elements of one tensor that a workgroup takes
constexpr int kAdamPointers = 400; // gradient pointers of one launch (they travel as kernel arguments)

// One tensor of an optimiser, in device memory.
struct AdamTensor {
  float* p;
  void* m;         // fp32, or 8-bit codes
  void* v;
  uint8_t* m_exp;  // 8 bits: one biased exponent per block
  uint8_t* v_exp;
  void* copy;      // or null
  int64_t n;
  uint32_t first;  // number of the first element, through all tensors (mod 2^32)
  int32_t wide;    // p, m, v and copy allow vector accesses from every eighth element
};

struct AdamChunk {
  int32_t tensor, index;  // elements [index * kAdamChunk, ...) of the tensor
};

struct AdamStep {
  const AdamTensor* tensors;
  const AdamChunk* chunks;   // of this launch's tensors
  int32_t first_tensor;
  float decay;               // lr weight_decay
  float rate;                // lr / (1 - beta1^t)
  float root_scale;          // 1 / sqrt(1 - beta2^t)
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  uint32_t salt;             // of the random bits: seed and step
  const void* grads[kAdamPointers];
};

struct AdamValues {
  const AdamTensor* tensors;
  const AdamChunk* chunks;
  int32_t first_tensor;
  void* out[kAdamPointers];  // m's and v's tensor in turn
};

hipError_t launch_adamw(const AdamStep& a, int64_t chunks, int state_bits, int grad_type, int copy_type, hipStream_t s);
hipError_t launch_adamw_values(const AdamValues& a, int64_t chunks, int state_bits, int type, hipStream_t s);

}  // namespace xtvxy
