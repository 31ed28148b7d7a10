// The AdamW step over many tensors in one launch, with states in 32 bits or in 8.
//
// Memory bound: an element moves 4 + 4 bytes of p, 2 or 4 of the gradient, 8 + 8 of 32-bit states or
// 2 + 2 (and 4 / 128) of 8-bit ones, and 2 of a 16-bit copy. A workgroup takes 2048 elements of one
// tensor, a thread 8 neighbours: 16-byte accesses of every operand but the 8-bit states (8 bytes), and
// a block of 128 elements, which shares an exponent, lies in 16 lanes. 100 M elements with bf16 gradients and
// copies: 518 us with 32-bit states (5.4 TB/s; a copy of 4 GiB reaches 4.7), 306 us with 8-bit ones
// (5.2 TB/s), and 113 us to write the values of both (5.3 TB/s).
#include "adamw.h"
#include "linear_util.h"

namespace xtvxy {
namespace {

constexpr int kThreads = 256;
static_assert(kThreads * 8 == kAdamChunk, "a thread takes eight elements");

// 32 bits that depend on the element's number and the salt: two rounds of multiply and xor-shift.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0xBB67AE85u;
  x = (x ^ (x >> 15)) * 0x3C6EF373u;
  return x ^ (x >> 16);
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int count, bool wide, float (&x)[8]) {
  if (wide && count == 8) {
    const typename Vec<T>::x8 v = *reinterpret_cast<const typename Vec<T>::x8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < count ? (float)p[i] : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int count, bool wide, const float (&x)[8]) {
  if (wide && count == 8) {
    typename Vec<T>::x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)x[i];
    *reinterpret_cast<typename Vec<T>::x8*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = (T)x[i];
  }
}

// Eight codes as two words, the first in the lowest byte; missing ones are zero.
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int count, bool wide) {
  if (wide && count == 8) return *reinterpret_cast<const u32x2*>(p);
  u32x2 r = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < count) r[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int count, bool wide, u32x2 c) {
  if (wide && count == 8) {
    *reinterpret_cast<u32x2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = (uint8_t)(c[i / 4] >> (8 * (i & 3)));
  }
}

// m's codes are e4m3 without infinities (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f is
// NaN). A code's bits shifted to an fp32's exponent and mantissa read as the value times 2^-120,
// subnormals included, so one exponent shift finishes the decoding.
__device__ __forceinline__ float decode_m(uint32_t code, int exponent) {
  const uint32_t mag = code & 0x7f;
  const float x = ldexpf(__uint_as_float(mag << 20), exponent - 127 + 120);
  const uint32_t sign = (code & 0x80) << 24;
  return mag == 0x7f ? __uint_as_float(0x7fc00000u) : __uint_as_float(__float_as_uint(x) | sign);
}
// v's codes have no sign, 4 exponent bits of bias 15 and 4 mantissa bits (0 .. 1.9375, subnormal steps
// of 2^-18): the same with 2^-112.
__device__ __forceinline__ float decode_v(uint32_t code, int exponent) {
  return ldexpf(__uint_as_float(code << 19), exponent - 127 + 112);
}

// Rounding at random: of the 20 (19) bits below a code's last, the random bits are added before they
// are cut off, so a value is rounded up with the probability of its remainder. The same shift as in
// decoding makes subnormal codes come out of fp32's subnormals.
__device__ __forceinline__ uint32_t encode_m(float m, int exponent, uint32_t rnd) {
  const float x = ldexpf(fabsf(m), 127 - exponent - 120);
  const uint32_t up = ((rnd >> 19) << 7) | 64u;
  uint32_t code = (__float_as_uint(x) + up) >> 20;
  code = __float_as_uint(x) >= 0x7f800000u ? 0x7fu : code;  // NaN and infinities: NaN
  return code | (m < 0.0f ? 0x80u : 0u);
}
__device__ __forceinline__ uint32_t encode_v(float v, int exponent, uint32_t rnd) {
  const float x = ldexpf(v, 127 - exponent - 112);
  uint32_t code = (__float_as_uint(x) + (rnd & 0x7ffffu)) >> 19;
  code = code > 255u ? 255u : code;  // NaN, infinities and what no exponent holds: the largest
  return v > 0.0f && code < 1u ? 1u : code;  // what is not zero is not stored as zero: m / sqrt(v) stays bounded
}

// The smallest biased exponent e in 1..253 with top <= limit 2^(e - 127 + shift), limit 1.mantissa.
__device__ __forceinline__ int block_exponent(uint32_t top_bits, uint32_t limit_mantissa, int shift) {
  const int e = (int)(top_bits >> 23) + ((top_bits & 0x7fffffu) > limit_mantissa ? 1 : 0) - shift;
  return min(max(e, 1), 253);
}

// The largest of x over the 16 lanes of a row.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)dpp_int<dpp::kXor1>(0, (int)x));
  x = max(x, (uint32_t)dpp_int<dpp::kXor2>(0, (int)x));
  x = max(x, (uint32_t)dpp_int<dpp::kHalfMirror>(0, (int)x));
  return max(x, (uint32_t)dpp_int<dpp::kMirror>(0, (int)x));
}
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(fabsf(x));
  return b < 0x7f800000u ? b : 0u;
}

// p - (decay p + update). A factor 1 - decay would be kept to steps of 6e-8 only: a decay of 2e-8 a step would be
// none, the same way for every element and step. An infinite p stays infinite.
__device__ __forceinline__ float moved(float p, float decay, float update) {
  return p - (fabsf(p) < INFINITY ? fmaf(decay, p, update) : update);
}

struct NoCopy {};
template <typename C>
struct CopyOut {
  static __device__ __forceinline__ void store(const AdamTensor& t, int64_t at, int count, const float (&x)[8]) {
    store8<C>(static_cast<C*>(t.copy) + at, count, t.wide, x);
  }
};
template <>
struct CopyOut<NoCopy> {
  static __device__ __forceinline__ void store(const AdamTensor&, int64_t, int, const float (&)[8]) {}
};

template <int kBits, typename G, typename C>
__global__ __launch_bounds__(kThreads) void adamw_step(AdamStep a) {
  const AdamChunk chunk = a.chunks[blockIdx.x];
  const AdamTensor t = a.tensors[chunk.tensor];
  const G* g = static_cast<const G*>(a.grads[chunk.tensor - a.first_tensor]);
  const int64_t at = (int64_t)chunk.index * kAdamChunk + threadIdx.x * 8;
  const int64_t left = t.n - at;
  const int count = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
  const bool wide = t.wide, wide_g = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
  float p[8], gr[8], m[8], v[8];
  u32x2 mc = {0, 0}, vc = {0, 0};
  const int64_t block = at / kAdamBlock;
  load8<float>(t.p + at, count, wide, p);
  load8<G>(g + at, count, wide_g, gr);
  if (kBits == 32) {
    load8<float>(static_cast<const float*>(t.m) + at, count, wide, m);
    load8<float>(static_cast<const float*>(t.v) + at, count, wide, v);
  } else {
    mc = load_codes(static_cast<const uint8_t*>(t.m) + at, count, wide);
    vc = load_codes(static_cast<const uint8_t*>(t.v) + at, count, wide);
    const int me = count > 0 ? t.m_exp[block] : 1, ve = count > 0 ? t.v_exp[block] : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = decode_m((mc[i / 4] >> (8 * (i & 3))) & 0xff, me);
      v[i] = decode_v((vc[i / 4] >> (8 * (i & 3))) & 0xff, ve);
    }
  }
  // The hardware's square root takes subnormals as zero (roots of up to 1.1e-19), half a unit of an eps of
  // 1.8e-12 times the root's factor; a smaller eps takes the library's square root and division.
  const bool exact = a.eps < 2e-12f * a.root_scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = fmaf(gr[i], a.one_minus_beta1, m[i] * a.beta1);
    // not through g^2, which leaves fp32 from 1.9e19 on
    v[i] = fmaf(gr[i] * a.one_minus_beta2, gr[i], v[i] * a.beta2);
  }
  if (exact) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = moved(p[i], a.decay, a.rate * m[i] / (sqrtf(v[i]) * a.root_scale + a.eps));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float root = __builtin_amdgcn_sqrtf(v[i]);
      p[i] = moved(p[i], a.decay, a.rate * m[i] * fast_rcp(fmaf(root, a.root_scale, a.eps)));
    }
  }
  store8<float>(t.p + at, count, wide, p);
  CopyOut<C>::store(t, at, count, p);
  if (kBits == 32) {
    store8<float>(static_cast<float*>(t.m) + at, count, wide, m);
    store8<float>(static_cast<float*>(t.v) + at, count, wide, v);
  } else {
    uint32_t mt = 0, vt = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // A finite gradient whose square leaves fp32: m / sqrt(v) is zero in this step, but v's code cannot say
      // infinity (and its block's exponent goes by the others), so m is dropped: the next step would take it
      // over the square root of a far smaller v.
      if (v[i] == INFINITY && fabsf(m[i]) < INFINITY) m[i] = 0.0f;
      mt = max(mt, finite_bits(m[i]));
      vt = max(vt, finite_bits(v[i]));
    }
    // elements that do not exist are zero and change no maximum
    const int me = block_exponent(row_max(mt), 0x600000u, 8);  // 448 = 1.75 * 2^8: holds all of fp32
    const int ve = block_exponent(row_max(vt), 0x780000u, 0);  // 1.9375
    u32x2 mo = {0, 0}, vo = {0, 0};
    uint32_t h = (t.first + (uint32_t)at) * 0x9E3779B1u + a.salt;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t rnd = mix(h);
      h += 0x9E3779B1u;
      mo[i / 4] |= encode_m(m[i], me, rnd) << (8 * (i & 3));
      vo[i / 4] |= encode_v(v[i], ve, rnd) << (8 * (i & 3));
    }
    store_codes(static_cast<uint8_t*>(t.m) + at, count, wide, mo);
    store_codes(static_cast<uint8_t*>(t.v) + at, count, wide, vo);
    if (count > 0 && (threadIdx.x & 15) == 0) {
      t.m_exp[block] = (uint8_t)me;
      t.v_exp[block] = (uint8_t)ve;
    }
  }
}

template <int kBits, typename T>
__global__ __launch_bounds__(kThreads) void adamw_values(AdamValues a) {
  const AdamChunk chunk = a.chunks[blockIdx.x];
  const AdamTensor t = a.tensors[chunk.tensor];
  T* mo = static_cast<T*>(a.out[2 * (chunk.tensor - a.first_tensor)]);
  T* vo = static_cast<T*>(a.out[2 * (chunk.tensor - a.first_tensor) + 1]);
  const int64_t at = (int64_t)chunk.index * kAdamChunk + threadIdx.x * 8;
  const int64_t left = t.n - at;
  if (left <= 0) return;
  const int count = left >= 8 ? 8 : (int)left;
  float m[8], v[8];
  if (kBits == 32) {
    load8<float>(static_cast<const float*>(t.m) + at, count, t.wide, m);
    load8<float>(static_cast<const float*>(t.v) + at, count, t.wide, v);
  } else {
    const u32x2 mc = load_codes(static_cast<const uint8_t*>(t.m) + at, count, t.wide);
    const u32x2 vc = load_codes(static_cast<const uint8_t*>(t.v) + at, count, t.wide);
    const int me = t.m_exp[at / kAdamBlock], ve = t.v_exp[at / kAdamBlock];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = decode_m((mc[i / 4] >> (8 * (i & 3))) & 0xff, me);
      v[i] = decode_v((vc[i / 4] >> (8 * (i & 3))) & 0xff, ve);
    }
  }
  store8<T>(mo + at, count, (reinterpret_cast<uintptr_t>(mo) & 15) == 0, m);
  store8<T>(vo + at, count, (reinterpret_cast<uintptr_t>(vo) & 15) == 0, v);
}

template <int kBits, typename G>
hipError_t step_for(const AdamStep& a, unsigned grid, int copy_type, hipStream_t s) {
  if (copy_type == kBf16) adamw_step<kBits, G, __bf16><<<grid, kThreads, 0, s>>>(a);
  else if (copy_type == kF16) adamw_step<kBits, G, _Float16><<<grid, kThreads, 0, s>>>(a);
  else adamw_step<kBits, G, NoCopy><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <int kBits>
hipError_t step_bits(const AdamStep& a, unsigned grid, int grad_type, int copy_type, hipStream_t s) {
  if (grad_type == kBf16) return step_for<kBits, __bf16>(a, grid, copy_type, s);
  if (grad_type == kF16) return step_for<kBits, _Float16>(a, grid, copy_type, s);
  return step_for<kBits, float>(a, grid, copy_type, s);
}

template <int kBits>
hipError_t values_bits(const AdamValues& a, unsigned grid, int type, hipStream_t s) {
  if (type == kBf16) adamw_values<kBits, __bf16><<<grid, kThreads, 0, s>>>(a);
  else if (type == kF16) adamw_values<kBits, _Float16><<<grid, kThreads, 0, s>>>(a);
  else adamw_values<kBits, float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(const AdamStep& a, int64_t chunks, int state_bits, int grad_type, int copy_type, hipStream_t s) {
  if (state_bits == 8) return step_bits<8>(a, (unsigned)chunks, grad_type, copy_type, s);
  return step_bits<32>(a, (unsigned)chunks, grad_type, copy_type, s);
}

hipError_t launch_adamw_values(const AdamValues& a, int64_t chunks, int state_bits, int type, hipStream_t s) {
  if (state_bits == 8) return values_bits<8>(a, (unsigned)chunks, type, s);
  return values_bits<32>(a, (unsigned)chunks, type, s);
}

}  // namespace xtvxy
