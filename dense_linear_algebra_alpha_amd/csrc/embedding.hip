// Embedding lookup out[i] = scale table[ids[i]] and its gradient dtable[r] = scale sum over ids[i] = r of G[i].
//
// Both are bound by memory: the lookup reads and writes a row per token; the gradient reads one per token and
// writes the whole table, most of it zeros.
//
// The gradient sorts the tokens by their row (a stable radix sort, 9 bits a pass or less), so that each row's sum is
// taken in the order of the tokens, in fp32, and rounded once: it is bitwise reproducible, and needs no atomics.
// Up to 16384 tokens one workgroup sorts in LDS; the other CUs write the table's zeros meanwhile. Beyond, each pass
// takes a launch that counts digits and one that places the tokens, and each writes its share of the zeros.
// Then a wavefront sums 32 sorted tokens over 1 KiB of their columns. A row whose tokens lie within the 32 is
// written at once; of rows that cross over, which frequent words have, the sums go to the workspace and a last launch
// joins them in order.
#include <utility>

#include "embedding.h"
#include "linear_util.h"

namespace xtvxy {
namespace {

template <typename T>
constexpr int kChunkOf = 16 / sizeof(T);

__device__ __forceinline__ int64_t index_at(const void* p, int bits, int64_t i) {
  return bits == 32 ? static_cast<const int32_t*>(p)[i] : static_cast<const int64_t*>(p)[i];
}

// 256 / kLanes tokens a workgroup, kLanes threads each. The last chunk of a row that is no whole number of
// chunks is its last 16 bytes, written twice in part. kNarrow: rows shorter than a chunk.
template <typename T, int kLanes, bool kNarrow>
__global__ __launch_bounds__(256) void embedding_rows(EmbeddingArgs a) {
  constexpr int V = kChunkOf<T>, kTokens = 256 / kLanes, kBatch = 4;
  const int t = threadIdx.x % kLanes;
  const int64_t chunks = (a.k + V - 1) / V;
  for (int64_t i = (int64_t)blockIdx.x * kTokens + threadIdx.x / kLanes; i < a.count; i += (int64_t)gridDim.x * kTokens) {
    const int64_t id = index_at(a.ids, a.index_bits, i);
    const bool there = id >= 0 && id < a.rows;
    const T* row = static_cast<const T*>(a.table) + (there ? id : 0) * a.ldt;
    T* out = static_cast<T*>(a.out) + i * a.ldo;
    const T otherwise = (T)(id < 0 ? 0.0f : __builtin_nanf(""));
    if (kNarrow) {
      for (int j = t; j < (int)a.k; j += kLanes) out[j] = there ? (T)((float)row[j] * a.scale) : otherwise;
      continue;
    }
    for (int64_t c0 = t; c0 < chunks; c0 += kLanes * kBatch) {
      T x[kBatch][V];
      int64_t at[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {  // beyond the row: its last chunk again
        const int64_t j = (c0 + b * kLanes) * V;
        at[b] = j < a.k - V ? j : a.k - V;
        if (there) __builtin_memcpy(x[b], row + at[b], 16);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (c0 + b * kLanes >= chunks) break;
        T o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = there ? (T)((float)x[b][e] * a.scale) : otherwise;
        __builtin_memcpy(out + at[b], o, 16);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the gradient: sorting
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kSortRounds = kSortItems / kSortThreads;

// The zeros of rows [first, end) of the table, by the workgroups from `groups` on.
struct Fill {
  char* p;
  int64_t pitch, row_bytes, first, end;
  int32_t element;
};

__device__ __forceinline__ void fill_rows(const Fill& f, int64_t group, int64_t groups) {
  const u32x4 zero = {0, 0, 0, 0};
  const int64_t rows = f.end - f.first;
  if (rows <= 0) return;
  if (f.pitch == f.row_bytes && f.row_bytes * rows >= 16) {  // one stretch of memory
    char* p = f.p + f.first * f.pitch;
    const int64_t bytes = rows * f.row_bytes, chunks = (bytes + 15) / 16;
    for (int64_t c = group * kSortThreads + threadIdx.x; c < chunks; c += groups * kSortThreads) {
      const int64_t at = c * 16 < bytes - 16 ? c * 16 : bytes - 16;
      __builtin_memcpy(p + at, &zero, 16);
    }
    return;
  }
  for (int64_t r = f.first + group; r < f.end; r += groups) {
    char* p = f.p + r * f.pitch;
    if (f.row_bytes >= 16) {
      for (int64_t at = threadIdx.x * 16; at < f.row_bytes; at += kSortThreads * 16)
        __builtin_memcpy(p + (at < f.row_bytes - 16 ? at : f.row_bytes - 16), &zero, 16);
    } else {
      for (int64_t at = threadIdx.x * f.element; at < f.row_bytes; at += kSortThreads * f.element)
        __builtin_memset(p + at, 0, f.element == 2 ? 2 : 4);
    }
  }
}

struct SortArgs {
  const void* ids;       // the keys of the first pass, else null
  int32_t index_bits;
  int64_t count, rows;
  const uint32_t* keys;  // of later passes
  const uint32_t* from;
  uint32_t* keys_out;
  uint32_t* from_out;
  uint32_t* counts;
  int32_t shift, bits, end_bit;  // this pass's digit; sort_all: up to end_bit
  int32_t groups;                // sorting workgroups; the others fill
  Fill fill;
};

__device__ __forceinline__ uint32_t key_of(const SortArgs& a, int64_t i) {
  if (!a.ids) return a.keys[i];
  const int64_t id = index_at(a.ids, a.index_bits, i);
  return id >= 0 && id < a.rows ? (uint32_t)id : (uint32_t)a.rows;
}

struct SortShared {
  uint32_t count[kSortWaves][kDigits];  // of each wavefront's keys by digit, then those of the wavefronts before
  uint32_t base[kDigits];               // of all keys with smaller digits
  uint32_t wave_total[kSortWaves];
};

// Each key's rank among its wavefront's keys of the same digit, in order; count[wave][digit] in the end. Keys of
// round r of wavefront w come after those of earlier rounds and wavefronts.
__device__ __forceinline__ void rank_keys(SortShared& s, const uint32_t (&key)[kSortRounds], uint32_t (&rank)[kSortRounds],
                                          int rounds, int shift, int bits) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  for (int d = threadIdx.x; d < kSortWaves * kDigits; d += kSortThreads) (&s.count[0][0])[d] = 0;
  __syncthreads();
  volatile uint32_t* count = s.count[wave];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    rank[r] = 0;
    if (r < rounds) {
      const uint32_t digit = (key[r] >> shift) & ((1u << bits) - 1);
      uint64_t same = ~(uint64_t)0;
#pragma unroll
      for (int b = 0; b < kDigitBits; ++b) {  // bits beyond the digit's are zero in every key
        const bool one = digit >> b & 1;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
      }
      const uint32_t before = __popcll(same & below), first = count[digit];
      rank[r] = first + before;
      __builtin_amdgcn_wave_barrier();
      if (before == 0) count[digit] = first + (uint32_t)__popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
}

// count[wave][digit] becomes the sum over earlier wavefronts, base[digit] the sum over smaller digits of `total`
// (of this workgroup's keys; with `counts`, of all workgroups') plus what earlier workgroups have of the digit.
__device__ __forceinline__ void place_digits(SortShared& s, const uint32_t* counts, int groups) {
  const int d = threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t total = 0, earlier = 0;
  if (d < kDigits) {
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = s.count[w][d];
      s.count[w][d] = total;
      total += c;
    }
    if (counts) {
      total = 0;
#pragma unroll 8
      for (int g = 0; g < groups; ++g) {
        const uint32_t c = counts[g * kDigits + d];
        if (g < (int)blockIdx.x) earlier += c;
        total += c;
      }
    }
  }
  uint32_t sum = total;  // inclusive over the wavefront's digits
  for (int by = 1; by < 64; by *= 2) {
    const uint32_t v = __shfl_up(sum, by);
    if (lane >= by) sum += v;
  }
  if (lane == 63) s.wave_total[wave] = sum;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < kDigits / 64; ++w)
    if (w < wave) before += s.wave_total[w];
  if (d < kDigits) s.base[d] = before + sum - total + earlier;
  __syncthreads();
}

// All passes in one workgroup: up to kSortItems keys. Padding keys are all ones and come last.
__global__ __launch_bounds__(kSortThreads) void sort_all(SortArgs a) {
  __shared__ SortShared s;
  __shared__ uint32_t keys[kSortItems];
  __shared__ uint16_t from[kSortItems];
  if ((int)blockIdx.x >= a.groups) return fill_rows(a.fill, blockIdx.x - a.groups, gridDim.x - a.groups);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, count = (int)a.count;
  const int rounds = (count + kSortThreads - 1) / kSortThreads;
  uint32_t key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int i = (wave * rounds + r) * 64 + lane;
    pos[r] = i;
    key[r] = r < rounds && i < count ? key_of(a, i) : ~0u;
  }
  for (int shift = 0; shift < a.end_bit; shift += a.bits) {
    rank_keys(s, key, rank, rounds, shift, a.bits);
    place_digits(s, nullptr, 1);
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (r < rounds) {
        const uint32_t digit = (key[r] >> shift) & ((1u << a.bits) - 1);
        const uint32_t to = s.base[digit] + s.count[wave][digit] + rank[r];
        keys[to] = key[r];
        from[to] = (uint16_t)pos[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (r < rounds) {
        const int i = (wave * rounds + r) * 64 + lane;
        key[r] = keys[i];
        pos[r] = from[i];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int i = (wave * rounds + r) * 64 + lane;
    if (r < rounds && i < count) {
      a.keys_out[i] = key[r];
      a.from_out[i] = pos[r];
    }
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_count(SortArgs a) {
  __shared__ uint32_t count[kDigits];
  if ((int)blockIdx.x >= a.groups) return fill_rows(a.fill, blockIdx.x - a.groups, gridDim.x - a.groups);
  if (threadIdx.x < kDigits) count[threadIdx.x] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kSortItems;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = first + r * kSortThreads + threadIdx.x;
    if (i < a.count) atomicAdd(&count[(key_of(a, i) >> a.shift) & ((1u << a.bits) - 1)], 1u);  // whole numbers: any order
  }
  __syncthreads();
  if (threadIdx.x < kDigits) a.counts[(int64_t)blockIdx.x * kDigits + threadIdx.x] = count[threadIdx.x];
}

__global__ __launch_bounds__(kSortThreads) void sort_place(SortArgs a) {
  __shared__ SortShared s;
  if ((int)blockIdx.x >= a.groups) return fill_rows(a.fill, blockIdx.x - a.groups, gridDim.x - a.groups);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t first = (int64_t)blockIdx.x * kSortItems;
  uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = first + (wave * kSortRounds + r) * 64 + lane;
    key[r] = i < a.count ? key_of(a, i) : ~0u;
  }
  rank_keys(s, key, rank, kSortRounds, a.shift, a.bits);
  place_digits(s, a.counts, a.groups);
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = first + (wave * kSortRounds + r) * 64 + lane;
    if (i >= a.count) continue;
    const uint32_t digit = (key[r] >> a.shift) & ((1u << a.bits) - 1);
    const uint32_t to = s.base[digit] + s.count[wave][digit] + rank[r];
    a.keys_out[to] = key[r];
    a.from_out[to] = a.from ? a.from[i] : (uint32_t)i;
  }
}

// ---------------------------------------------------------------------------
// the gradient: sums
// ---------------------------------------------------------------------------

// A lane's V columns of the row `key`: the sum rounded, on top of what is there where the caller accumulates.
// The first `skip` belong to the neighbour before (V: all of them).
template <typename T, int V>
__device__ __forceinline__ void write_row(const EmbeddingGradientArgs& a, uint32_t key, int64_t at, int skip, const float (&sum)[V]) {
  if (skip == V) return;
  T* p = static_cast<T*>(a.dtable) + (int64_t)key * a.lddt + at;
  T o[V];
  if (skip == 0) {
    if (a.accumulate) __builtin_memcpy(o, p, 16);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = (T)(a.accumulate ? fmaf(sum[e], a.scale, (float)o[e]) : sum[e] * a.scale);
    __builtin_memcpy(p, o, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e >= skip) p[e] = (T)(a.accumulate ? fmaf(sum[e], a.scale, (float)p[e]) : sum[e] * a.scale);
  }
}

// Where a lane's V columns of slab `slab` begin and how many of them it shares; false where there are none.
template <int V, bool kNarrow>
__device__ __forceinline__ bool lane_columns(int64_t k, int64_t slab, int64_t* at, int* skip) {
  const int64_t j = (slab * 64 + (threadIdx.x & 63)) * V, last = kNarrow ? 0 : k - V;
  *at = j < last ? j : last;
  *skip = j < last ? 0 : j - last < V ? (int)(j - last) : V;
  return *skip < V;
}

template <typename T, int V, bool kNarrow>
__device__ __forceinline__ void load_row(const T* p, int64_t k, T (&x)[V]) {
  if (!kNarrow) {
    __builtin_memcpy(x, p, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = e < (int)k ? p[e] : (T)0.0f;
  }
}

constexpr int kSumBatch = 8;  // rows under way

// kNarrow: rows shorter than a chunk, which lane 0 has alone.
template <typename T, bool kNarrow>
__global__ __launch_bounds__(256) void embedding_sums(EmbeddingGradientArgs a, int64_t pieces, int64_t slabs) {
  constexpr int V = kChunkOf<T>;
  const int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= pieces * slabs) return;
  const int64_t piece = task / slabs, slab = task % slabs, s0 = piece * kPieceTokens;
  const int lane = threadIdx.x & 63;
  const uint32_t none = (uint32_t)a.rows;
  // lanes 0 .. 31: the piece; lane 32: the token after; lane 63: the one before
  const int64_t i = lane == 63 ? s0 - 1 : s0 + (lane <= kPieceTokens ? lane : kPieceTokens);
  const uint32_t key = i >= 0 && i < a.count ? a.keys[0][i] : none;
  const uint32_t from = i >= 0 && i < a.count ? a.from[0][i] : 0;
  const int tokens = __popcll(__ballot(lane < kPieceTokens && key < none));  // those without a row come last
  if (tokens == 0) return;
  int64_t at;
  int skip;
  lane_columns<V, kNarrow>(a.k, slab, &at, &skip);
  if (kNarrow && skip < V) skip = 0;
  const T* G = static_cast<const T*>(a.g) + at;
  float sum[V] = {};
  bool crosses = __builtin_amdgcn_readlane(key, 63) == __builtin_amdgcn_readlane(key, 0);  // the first row began earlier
  const bool on = tokens == kPieceTokens;
  for (int j0 = 0; j0 < tokens; j0 += kSumBatch) {
    T x[kSumBatch][V];
#pragma unroll
    for (int b = 0; b < kSumBatch; ++b) {
      const int j = j0 + b < tokens ? j0 + b : tokens - 1;
      load_row<T, V, kNarrow>(G + (int64_t)(uint32_t)__builtin_amdgcn_readlane(from, j) * a.ldg, a.k, x[b]);
    }
#pragma unroll
    for (int b = 0; b < kSumBatch; ++b) {
      const int j = j0 + b;
      if (j >= tokens) break;
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] += (float)x[b][e];
      const uint32_t row = __builtin_amdgcn_readlane(key, j);
      const bool same = (uint32_t)__builtin_amdgcn_readlane(key, j + 1) == row, last = j + 1 == tokens;
      if (same && !last) continue;
      const bool goes_on = same && last && on;
      if (crosses || goes_on) {
        float* p = a.partial + ((piece * 2 + (crosses ? 0 : 1)) * slabs + slab) * (64 * V) + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 4) *reinterpret_cast<f32x4*>(p + e) = {sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
      } else if (kNarrow) {
        T* p = static_cast<T*>(a.dtable) + (int64_t)row * a.lddt;
        if (lane == 0)
          for (int e = 0; e < (int)a.k; ++e) p[e] = (T)(a.accumulate ? fmaf(sum[e], a.scale, (float)p[e]) : sum[e] * a.scale);
      } else {
        write_row<T, V>(a, row, at, skip, sum);
      }
      crosses = false;
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] = 0.0f;
    }
  }
}

// The rows that begin in a piece and go on in the next: slot 1 of that piece, then slot 0 of those that follow,
// in order. Four wavefronts share the pieces that follow: each adds every fourth one, the four sums join in LDS.
template <typename T, bool kNarrow>
__global__ __launch_bounds__(256) void embedding_join(EmbeddingGradientArgs a, int64_t pieces, int64_t slabs) {
  constexpr int V = kChunkOf<T>;
  __shared__ float join[4][64][V + 1];
  const int64_t piece = blockIdx.x / slabs, slab = blockIdx.x % slabs, end = (piece + 1) * kPieceTokens;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t none = (uint32_t)a.rows;
  const uint32_t* keys = a.keys[0];
  if (end >= a.count) return;
  const uint32_t key = keys[end - 1];
  if (key >= none || keys[end] != key) return;  // no row goes on
  const int64_t start = piece * kPieceTokens;
  if (start > 0 && keys[start] == key && keys[start - 1] == key) return;  // it began earlier
  const float* partial = a.partial + slab * (64 * V) + lane * V;
  const int64_t slot = slabs * (64 * V);
  float sum[V] = {};
  const auto add = [&](int64_t at) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(partial + at * slot + e);
#pragma unroll
      for (int x = 0; x < 4; ++x) sum[e + x] += p[x];
    }
  };
  if (wave == 0) add(piece * 2 + 1);
  for (int64_t q0 = piece + 1;; q0 += 64) {  // 64 pieces at a time: lane l looks whether the row goes on behind piece q0 + l
    const int64_t next = (q0 + lane + 1) * kPieceTokens;
    const uint64_t stops = __ballot(next >= a.count || keys[next < a.count ? next : 0] != key);
    const int more = stops ? __builtin_ctzll(stops) + 1 : 64;
#pragma unroll 8
    for (int q = wave; q < more; q += 4) add((q0 + q) * 2);
    if (stops) break;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) join[wave][lane][e] = sum[e];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < 4; ++w)
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] += join[w][lane][e];
  if (kNarrow) {
    T* p = static_cast<T*>(a.dtable) + (int64_t)key * a.lddt;
    if (lane == 0)
      for (int e = 0; e < (int)a.k; ++e) p[e] = (T)(a.accumulate ? fmaf(sum[e], a.scale, (float)p[e]) : sum[e] * a.scale);
    return;
  }
  int64_t at;
  int skip;
  lane_columns<V, kNarrow>(a.k, slab, &at, &skip);
  write_row<T, V>(a, key, at, skip, sum);
}

template <typename T>
void embedding_for(const EmbeddingArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  const int64_t chunks = (a.k + V - 1) / V;
  const auto grid = [&](int lanes) {
    const int64_t groups = (a.count * lanes + 255) / 256, most = (int64_t)1 << 22;
    return (unsigned)(groups < most ? groups : most);
  };
  if (a.k < V) embedding_rows<T, 4, true><<<grid(4), 256, 0, s>>>(a);
  else if (chunks <= 16) embedding_rows<T, 16, false><<<grid(16), 256, 0, s>>>(a);
  else if (chunks <= 256) embedding_rows<T, 64, false><<<grid(64), 256, 0, s>>>(a);
  else embedding_rows<T, 256, false><<<grid(256), 256, 0, s>>>(a);
}

template <typename T>
void sums_for(const EmbeddingGradientArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  const int64_t pieces = piece_count(a.count), slabs = (a.k + 64 * V - 1) / (64 * V);
  const unsigned groups = (unsigned)((pieces * slabs + 3) / 4);
  if (a.k < V) {
    embedding_sums<T, true><<<groups, 256, 0, s>>>(a, pieces, slabs);
    if (pieces > 1) embedding_join<T, true><<<(unsigned)(pieces * slabs), 256, 0, s>>>(a, pieces, slabs);
  } else {
    embedding_sums<T, false><<<groups, 256, 0, s>>>(a, pieces, slabs);
    if (pieces > 1) embedding_join<T, false><<<(unsigned)(pieces * slabs), 256, 0, s>>>(a, pieces, slabs);
  }
}

}  // namespace

hipError_t launch_embedding(const EmbeddingArgs& a, int type, hipStream_t s) {
  if (type == kBf16) embedding_for<__bf16>(a, s);
  else if (type == kF16) embedding_for<_Float16>(a, s);
  else embedding_for<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_embedding_gradient(const EmbeddingGradientArgs& args, int type, hipStream_t s) {
  EmbeddingGradientArgs a = args;
  SortArgs q{};
  q.index_bits = a.index_bits;
  q.count = a.count;
  q.rows = a.rows;
  q.counts = a.counts;
  q.groups = (int32_t)sort_groups(a.count);
  const int es = elem_size(type);
  q.fill = {static_cast<char*>(a.dtable), a.lddt * es, a.k * es, 0, 0, es};
  int bits = 1;
  while (bits < 32 && (uint64_t)a.rows >> bits) ++bits;
  const int passes = (bits + kDigitBits - 1) / kDigitBits;
  q.bits = (bits + passes - 1) / passes;
  const int steps = q.groups <= 1 ? 1 : 2 * passes;
  const int fillers = a.accumulate ? 0 : 512;
  for (int step = 0; step < steps; ++step) {
    q.fill.first = a.accumulate ? 0 : a.rows * step / steps;
    q.fill.end = a.accumulate ? 0 : a.rows * (step + 1) / steps;
    const unsigned grid = (unsigned)(q.groups + fillers);
    if (grid == 0) return hipSuccess;
    const int pass = step / 2, to = pass & 1;
    q.ids = pass == 0 ? a.ids : nullptr;
    q.keys = pass == 0 ? nullptr : a.keys[to ^ 1];
    q.from = pass == 0 ? nullptr : a.from[to ^ 1];
    q.keys_out = a.keys[to];
    q.from_out = a.from[to];
    q.shift = pass * q.bits;
    q.end_bit = bits;
    if (q.groups <= 1) sort_all<<<grid, kSortThreads, 0, s>>>(q);
    else if (step % 2 == 0) sort_count<<<grid, kSortThreads, 0, s>>>(q);
    else sort_place<<<grid, kSortThreads, 0, s>>>(q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.count == 0) return hipSuccess;
  if (q.groups > 1 && (passes - 1) % 2 == 1) {
    std::swap(a.keys[0], a.keys[1]);
    std::swap(a.from[0], a.from[1]);
  }
  if (type == kBf16) sums_for<__bf16>(a, s);
  else if (type == kF16) sums_for<_Float16>(a, s);
  else sums_for<float>(a, s);
  return hipGetLastError();
}

}  // namespace xtvxy
