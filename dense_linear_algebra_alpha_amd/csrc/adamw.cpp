// Host side of the AdamW step: the optimiser object (its tensors' table in device memory), argument
// checks and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "adamw.h"

using namespace xtvxy;

struct xtvxy_adamw_s {
  int device = 0;
  int32_t tensors = 0, state_bits = 32, copy_type = XTVXY_TYPE_NONE;
  std::vector<int64_t> numel;
  std::vector<int64_t> first_chunk;  // [tensors + 1]
  // what a step writes, as sorted disjoint [begin, end) byte ranges
  std::vector<std::pair<uintptr_t, uintptr_t>> written;
  AdamTensor* d_tensors = nullptr;
  AdamChunk* d_chunks = nullptr;

  ~xtvxy_adamw_s() {
    if (d_tensors) (void)hipFree(d_tensors);
    if (d_chunks) (void)hipFree(d_chunks);
  }
  // Whether a step writes into [begin, end). *at: how many ranges begin at or before the last address
  // asked for; lists mostly come in the order of their addresses, or lie between the same two ranges, and
  // then need no search (200 tensors: 2 us of a step's 9).
  bool writes(uintptr_t begin, uintptr_t end, size_t* at) const {
    size_t i = *at;
    if ((i > 0 && written[i - 1].first > begin) || (i < written.size() && written[i].first <= begin)) {
      i = std::upper_bound(written.begin(), written.end(), std::make_pair(begin, UINTPTR_MAX)) - written.begin();
      *at = i;
    }
    return (i < written.size() && written[i].first < end) || (i > 0 && written[i - 1].second > begin);
  }
};

namespace {

constexpr int64_t kMaxChunks = ((int64_t)1 << 24) - 1;  // workgroups of 256 threads in one launch

bool valid_type(int t) { return t == XTVXY_TYPE_F32 || t == XTVXY_TYPE_BF16 || t == XTVXY_TYPE_F16; }
int type_size(int t) { return t == XTVXY_TYPE_F32 ? 4 : 2; }
int elem_type(int t) { return t == XTVXY_TYPE_BF16 ? kBf16 : t == XTVXY_TYPE_F16 ? kF16 : kF32; }

bool on_its_device(const xtvxy_adamw_s* h) {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess && dev == h->device;
}

// Whether any two of the [begin, end) ranges overlap; sorts them.
bool overlap_within(std::vector<std::pair<uintptr_t, uintptr_t>>* ranges) {
  std::sort(ranges->begin(), ranges->end());
  for (size_t i = 1; i < ranges->size(); ++i)
    if ((*ranges)[i].first < (*ranges)[i - 1].second) return true;
  return false;
}

xtvxy_status create(int32_t tensors, const int64_t* numel, float* const* params, int state_bits, void* const* m,
                    void* const* v, uint8_t* const* m_exp, uint8_t* const* v_exp, int copy_type, void* const* copies,
                    xtvxy_adamw* out) {
  if (!out) return XTVXY_ERROR_NULL_POINTER;
  *out = nullptr;
  if (tensors < 0 || (state_bits != 32 && state_bits != 8)) return XTVXY_ERROR_INVALID_VALUE;
  const bool copy = copy_type != XTVXY_TYPE_NONE;
  if (copy && copy_type != XTVXY_TYPE_BF16 && copy_type != XTVXY_TYPE_F16) return XTVXY_ERROR_INVALID_VALUE;
  const bool q = state_bits == 8;
  if (tensors > 0 && (!numel || !params || !m || !v || (q && (!m_exp || !v_exp)) || (copy && !copies)))
    return XTVXY_ERROR_NULL_POINTER;
  xtvxy_adamw_s* h = new (std::nothrow) xtvxy_adamw_s;
  if (!h) return XTVXY_ERROR_LAUNCH;
  struct Guard {
    xtvxy_adamw_s* h;
    ~Guard() { delete h; }
  } guard{h};
  std::vector<AdamTensor> table((size_t)tensors);
  std::vector<AdamChunk> chunks;
  uint64_t number = 0;
  h->first_chunk.push_back(0);
  int64_t total = 0;
  for (int32_t i = 0; i < tensors; ++i) {
    const int64_t n = numel[i];
    if (n < 0 || n > ((int64_t)1 << 42)) return XTVXY_ERROR_INVALID_VALUE;
    total += (n + kAdamChunk - 1) / kAdamChunk;
    if (total > ((int64_t)1 << 31)) return XTVXY_ERROR_UNSUPPORTED;
    if ((n + kAdamChunk - 1) / kAdamChunk > kMaxChunks) return XTVXY_ERROR_UNSUPPORTED;
    if (n > 0 && (!params[i] || !m[i] || !v[i] || (q && (!m_exp[i] || !v_exp[i])) || (copy && !copies[i])))
      return XTVXY_ERROR_NULL_POINTER;
    AdamTensor& t = table[i];
    t.p = params[i];
    t.m = m[i];
    t.v = v[i];
    t.m_exp = q ? m_exp[i] : nullptr;
    t.v_exp = q ? v_exp[i] : nullptr;
    t.copy = copy ? copies[i] : nullptr;
    t.n = n;
    t.first = (uint32_t)number;
    const uintptr_t states = reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v);
    t.wide = (reinterpret_cast<uintptr_t>(t.p) | reinterpret_cast<uintptr_t>(t.copy)) % 16 == 0 &&
             states % (q ? 8 : 16) == 0;
    if ((reinterpret_cast<uintptr_t>(t.p) | (q ? 0 : states)) % 4 != 0 || reinterpret_cast<uintptr_t>(t.copy) % 2 != 0)
      return XTVXY_ERROR_INVALID_VALUE;
    const int64_t blocks = (n + kAdamBlock - 1) / kAdamBlock;
    number += (uint64_t)blocks * kAdamBlock;
    for (int64_t c = 0; c * kAdamChunk < n; ++c) chunks.push_back({i, (int32_t)c});
    h->numel.push_back(n);
    h->first_chunk.push_back((int64_t)chunks.size());
    auto add = [&](const void* p, int64_t bytes) {
      if (p && bytes > 0) h->written.emplace_back(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes);
    };
    add(t.p, n * 4);
    add(t.m, n * (q ? 1 : 4));
    add(t.v, n * (q ? 1 : 4));
    add(t.m_exp, blocks);
    add(t.v_exp, blocks);
    add(t.copy, n * 2);
  }
  if (overlap_within(&h->written)) return XTVXY_ERROR_ALIASING;
  h->tensors = tensors;
  h->state_bits = state_bits;
  h->copy_type = copy_type;
  if (hipGetDevice(&h->device) != hipSuccess) return XTVXY_ERROR_LAUNCH;
  if (!chunks.empty()) {
    if (hipMalloc(&h->d_tensors, table.size() * sizeof(AdamTensor)) != hipSuccess ||
        hipMalloc(&h->d_chunks, chunks.size() * sizeof(AdamChunk)) != hipSuccess ||
        hipMemcpy(h->d_tensors, table.data(), table.size() * sizeof(AdamTensor), hipMemcpyHostToDevice) != hipSuccess ||
        hipMemcpy(h->d_chunks, chunks.data(), chunks.size() * sizeof(AdamChunk), hipMemcpyHostToDevice) != hipSuccess)
      return XTVXY_ERROR_LAUNCH;
  }
  guard.h = nullptr;
  *out = h;
  return XTVXY_SUCCESS;
}

// Calls fn(first tensor, tensors, first chunk, chunks) for runs of at most `most` tensors and
// kMaxChunks chunks.
template <typename F>
xtvxy_status for_runs(const xtvxy_adamw_s* h, int most, F fn) {
  for (int32_t t0 = 0; t0 < h->tensors;) {
    int32_t t1 = t0 + 1;
    while (t1 < h->tensors && t1 - t0 < most && h->first_chunk[t1 + 1] - h->first_chunk[t0] <= kMaxChunks) ++t1;
    const int64_t c0 = h->first_chunk[t0], c1 = h->first_chunk[t1];
    if (c1 > c0 && fn(t0, t1, c0, c1 - c0) != hipSuccess) return XTVXY_ERROR_LAUNCH;
    t0 = t1;
  }
  return XTVXY_SUCCESS;
}

xtvxy_status state_values(const xtvxy_adamw_s* h, void* const* m_out, void* const* v_out, int type, hipStream_t stream) {
  if (!h) return XTVXY_ERROR_NULL_POINTER;
  if (!valid_type(type)) return XTVXY_ERROR_INVALID_VALUE;
  if (h->first_chunk.back() == 0) return XTVXY_SUCCESS;
  if (!m_out || !v_out) return XTVXY_ERROR_NULL_POINTER;
  const int es = type_size(type);
  std::vector<std::pair<uintptr_t, uintptr_t>> out;
  out.reserve(2 * h->numel.size());
  size_t at = 0;
  for (int32_t i = 0; i < h->tensors; ++i) {
    if (h->numel[i] == 0) continue;
    for (const void* p : {m_out[i], v_out[i]}) {
      const uintptr_t o = reinterpret_cast<uintptr_t>(p);
      if (!o) return XTVXY_ERROR_NULL_POINTER;
      if (o % es != 0) return XTVXY_ERROR_INVALID_VALUE;
      const uintptr_t end = o + (uintptr_t)h->numel[i] * es;
      if (h->writes(o, end, &at)) return XTVXY_ERROR_ALIASING;
      out.emplace_back(o, end);
    }
  }
  if (overlap_within(&out)) return XTVXY_ERROR_ALIASING;
  if (!on_its_device(h)) return XTVXY_ERROR_INVALID_VALUE;
  AdamValues a;
  a.tensors = h->d_tensors;
  return for_runs(h, kAdamPointers / 2, [&](int32_t t0, int32_t t1, int64_t c0, int64_t chunks) {
    a.chunks = h->d_chunks + c0;
    a.first_tensor = t0;
    for (int32_t i = t0; i < t1; ++i) {
      a.out[2 * (i - t0)] = m_out[i];
      a.out[2 * (i - t0) + 1] = v_out[i];
    }
    return launch_adamw_values(a, chunks, h->state_bits, elem_type(type), stream);
  });
}

}  // namespace

extern "C" {

xtvxy_status xtvxy_adamw_create(int32_t tensors, const int64_t* numel, float* const* params, int state_bits,
                                void* const* m, void* const* v, uint8_t* const* m_exp, uint8_t* const* v_exp,
                                int copy_type, void* const* copies, xtvxy_adamw* optimiser) {
  try {
    return create(tensors, numel, params, state_bits, m, v, m_exp, v_exp, copy_type, copies, optimiser);
  } catch (const std::exception&) {  // host memory
    return XTVXY_ERROR_LAUNCH;
  }
}

xtvxy_status xtvxy_adamw_destroy(xtvxy_adamw optimiser) {
  delete optimiser;
  return XTVXY_SUCCESS;
}

xtvxy_status xtvxy_adamw_step(xtvxy_adamw h, const void* const* grads, int grad_type, int64_t step, double lr,
                              double beta1, double beta2, double eps, double weight_decay, uint32_t seed,
                              hipStream_t stream) {
  if (!h) return XTVXY_ERROR_NULL_POINTER;
  if (!valid_type(grad_type) || step < 1 || !(lr >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
      !(eps >= 0) || !(weight_decay >= 0) || !std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(weight_decay))
    return XTVXY_ERROR_INVALID_VALUE;
  if (h->first_chunk.back() == 0) return XTVXY_SUCCESS;
  if (!grads) return XTVXY_ERROR_NULL_POINTER;
  const int es = type_size(grad_type);
  size_t at = 0;
  for (int32_t i = 0; i < h->tensors; ++i) {
    if (h->numel[i] == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
    if (!g) return XTVXY_ERROR_NULL_POINTER;
    if (g % es != 0) return XTVXY_ERROR_INVALID_VALUE;
    if (h->writes(g, g + (uintptr_t)h->numel[i] * es, &at)) return XTVXY_ERROR_ALIASING;
  }
  if (!on_its_device(h)) return XTVXY_ERROR_INVALID_VALUE;
  AdamStep a;
  a.tensors = h->d_tensors;
  a.decay = (float)(lr * weight_decay);
  a.rate = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  a.root_scale = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  a.beta1 = (float)beta1;
  a.one_minus_beta1 = (float)(1.0 - beta1);
  a.beta2 = (float)beta2;
  a.one_minus_beta2 = (float)(1.0 - beta2);
  a.eps = (float)eps;
  a.salt = seed * 0xBB67AE85u + (uint32_t)step * 0x3C6EF373u;
  return for_runs(h, kAdamPointers, [&](int32_t t0, int32_t t1, int64_t c0, int64_t chunks) {
    a.chunks = h->d_chunks + c0;
    a.first_tensor = t0;
    std::copy(grads + t0, grads + t1, a.grads);
    return launch_adamw(a, chunks, h->state_bits, elem_type(grad_type),
                        h->copy_type == XTVXY_TYPE_NONE ? -1 : elem_type(h->copy_type), stream);
  });
}

xtvxy_status xtvxy_adamw_state_values(xtvxy_adamw optimiser, void* const* m_out, void* const* v_out, int type,
                                      hipStream_t stream) {
  try {
    return state_values(optimiser, m_out, v_out, type, stream);
  } catch (const std::exception&) {  // host memory
    return XTVXY_ERROR_LAUNCH;
  }
}

}  // extern "C"
