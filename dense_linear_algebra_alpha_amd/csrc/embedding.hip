// Embedding lookup out[i] = scale table[ids[i]] and its gradient dtable[r] = scale sum over ids[i] = r of G[i].
//
// Both are bound by memory: the lookup reads and writes a row per token; the gradient reads one per token and
// writes the whole table, most of it zeros.
//
// The gradient sorts the tokens by their row (a stable radix sort, 9 bits a pass or less), so that each row's sum is
// taken in the order of the tokens, in fp32, and rounded once: it is bitwise reproducible, and needs no atomics.
// Up to 4096 tokens one workgroup sorts in LDS. Beyond, each pass is a launch, beyond 32768 tokens one that counts
// digits and one that places the tokens. Meanwhile the other CUs write the table's zeros, each launch its share of them.
// Then a wavefront sums a piece of the sorted tokens over 1 KiB of their columns. A row whose tokens lie within the
// piece is written at once; of rows that cross over, which frequent words have, the sums go to the workspace and a last launch
// joins them in order.
//
// us of the kernels: lookup of 16384 tokens in 65536 x 4096 of bf16 32 (8.5 TB/s of rows read and written, 6.8 at memory); its
// gradient with 16384 tokens, 50001 x 2048: two sorting passes with the zeros of 205 MB 37 (5.5 TB/s), sums 20, join 6; 1777
// fp16 tokens of 1111 added to 10007 rows: sort 7, sums 8, join 4.5, each of them a launch and its chain of loads.
#include <type_traits>
#include <utility>

#include "embedding.h"
#include "linear_util.h"

namespace xtvxy {
namespace {

template <typename T>
constexpr int kChunkOf = 16 / sizeof(T);

typedef u32x4 unaligned_chunk __attribute__((aligned(2)));

__device__ __forceinline__ int64_t index_at(const void* p, int bits, int64_t i) {
  return bits == 32 ? static_cast<const int32_t*>(p)[i] : static_cast<const int64_t*>(p)[i];
}

template <bool kStreamed>
__device__ __forceinline__ void store_chunk(void* p, u32x4 v) {
  if (kStreamed) __builtin_nontemporal_store(v, static_cast<unaligned_chunk*>(p));
  else __builtin_memcpy(p, &v, 16);
}

// 256 / kLanes tokens a workgroup, kLanes threads each. The last chunk of a row that is no whole number of
// chunks is its last 16 bytes, written twice in part. kNarrow: rows shorter than a chunk. kStreamed: outputs beyond the
// L2s are stored past them, so that rows of the table that occur again stay there (16384 tokens x 4096 of bf16: 47
// to 35 us; with 256 threads and two chunks each in place of 64 and eight 32 us, 5.8 TB/s).
template <typename T, int kLanes, bool kNarrow, bool kStreamed>
__global__ __launch_bounds__(256) void embedding_rows(EmbeddingArgs a) {
  constexpr int V = kChunkOf<T>, kTokens = 256 / kLanes, kBatch = 2;
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
        u32x4 v;
        __builtin_memcpy(&v, o, 16);
        store_chunk<kStreamed>(out + at[b], v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the gradient: sorting
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024;

// The zeros of rows [first, end) of the table, by the workgroups from `groups` on, past the L2s (us: 50001 x 2048 of bf16 76 to
// 70, 184502 x 1186 of fp32 311 to 302; tables of up to 66 MB the same).
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
    const int64_t bytes = rows * f.row_bytes, chunks = (bytes + 15) / 16, step = groups * kSortThreads;
    int64_t c = group * kSortThreads + threadIdx.x;
    for (; c + 7 * step < chunks - 1; c += 8 * step) {
#pragma unroll
      for (int u = 0; u < 8; ++u) store_chunk<true>(p + (c + u * step) * 16, zero);
    }
    for (; c < chunks; c += step) __builtin_memcpy(p + (c < chunks - 1 ? c * 16 : bytes - 16), &zero, 16);
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

typedef __attribute__((address_space(3))) uint32_t lds_word;
constexpr int kSortWaves = kSortThreads / 64;

struct SortShared {
  uint32_t count[kSortWaves][kDigits];  // of each wavefront's keys by digit, then those of the wavefronts before
  uint32_t base[kDigits];               // where the workgroup's first key of the digit goes
  uint32_t total[kDigits], before[kDigits];  // keys of the digit, and those before the workgroup's
  uint32_t wave_total[kSortWaves];
};

// The sum of x over the threads before this one; `totals`: a word of LDS for each wavefront.
__device__ __forceinline__ uint32_t sum_before(uint32_t x, uint32_t* totals) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t sum = x;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) {
    const uint32_t v = __shfl_up(sum, by);
    if (lane >= by) sum += v;
  }
  if (lane == 63) totals[wave] = sum;
  __syncthreads();
  uint32_t before = sum - x;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w)
    if (w < wave) before += totals[w];
  return before;
}

// Each key's rank among its wavefront's keys of the same digit, in order; count[wave][digit] in the end. Keys of round
// r of a wavefront come after those of earlier rounds and wavefronts. The lanes of a digit find each other bit by bit.
template <int kRounds>
__device__ __forceinline__ void rank_keys(SortShared& s, const uint32_t (&key)[kRounds], uint32_t (&rank)[kRounds], int shift, int bits) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  for (int d = threadIdx.x; d < kSortWaves * kDigits; d += kSortThreads) (&s.count[0][0])[d] = 0;
  __syncthreads();
  // LDS by its own instructions (a generic pointer would wait for memory as well); in order within a wavefront
  volatile lds_word* count = (volatile lds_word*)s.count[wave];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
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
  __syncthreads();
}

// base from total and before (or, where the workgroup has all keys, from its own counts), and the wavefronts' counts
// made those of earlier wavefronts.
__device__ __forceinline__ void place_digits(SortShared& s, bool alone) {
  const int d = threadIdx.x;
  uint32_t own = 0;
  if (d < kDigits) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = s.count[w][d];
      s.count[w][d] = own;
      own += c;
    }
  }
  const uint32_t total = d < kDigits ? (alone ? own : s.total[d]) : 0;
  const uint32_t smaller = sum_before(total, s.wave_total);
  if (d < kDigits) s.base[d] = smaller + (alone ? 0 : s.before[d]);
  __syncthreads();
}

// All passes in one workgroup: up to 1024 kRounds keys, of which each round takes 0.75 us a pass. Padding keys are all ones
// and come last.
template <int kRounds>
__global__ __launch_bounds__(kSortThreads) void sort_all(SortArgs a) {
  __shared__ SortShared s;
  __shared__ uint32_t keys[kRounds * kSortThreads], from[kRounds * kSortThreads];
  if ((int)blockIdx.x >= a.groups) return fill_rows(a.fill, blockIdx.x - a.groups, gridDim.x - a.groups);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const auto item = [&](int r) { return (wave * kRounds + r) * 64 + lane; };
  uint32_t key[kRounds], pos[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    pos[r] = item(r);
    key[r] = item(r) < a.count ? key_of(a, item(r)) : ~0u;
  }
  for (int shift = 0; shift < a.end_bit; shift += a.bits) {
    rank_keys<kRounds>(s, key, rank, shift, a.bits);
    place_digits(s, true);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const uint32_t digit = (key[r] >> shift) & ((1u << a.bits) - 1);
      const uint32_t to = s.base[digit] + s.count[wave][digit] + rank[r];
      keys[to] = key[r];
      from[to] = pos[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      key[r] = keys[item(r)];
      pos[r] = from[item(r)];
    }
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (item(r) < a.count) {
      a.keys_out[item(r)] = key[r];
      a.from_out[item(r)] = pos[r];
    }
  }
}

// Counters in eight copies, one for each of eight lanes: the high digits of frequent rows are alike, and additions to
// one word of LDS wait for each other (16384 tokens, one copy: 21 us a pass).
constexpr int kCopies = 8;

__global__ __launch_bounds__(kSortThreads) void sort_count(SortArgs a) {
  __shared__ uint32_t count[kCopies][kDigits];
  if ((int)blockIdx.x >= a.groups) return fill_rows(a.fill, blockIdx.x - a.groups, gridDim.x - a.groups);
  for (int d = threadIdx.x; d < kCopies * kDigits; d += kSortThreads) (&count[0][0])[d] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kCountedTile;
#pragma unroll
  for (int r = 0; r < kCountedTile / kSortThreads; ++r) {
    const int64_t i = first + r * kSortThreads + threadIdx.x;
    if (i < a.count)  // whole numbers: any order
      atomicAdd(&count[threadIdx.x % kCopies][(key_of(a, i) >> a.shift) & ((1u << a.bits) - 1)], 1u);
  }
  __syncthreads();
  if (threadIdx.x >= kDigits) return;
  uint32_t total = 0;
  for (int c = 0; c < kCopies; ++c) total += count[c][threadIdx.x];
  a.counts[(int64_t)blockIdx.x * kDigits + threadIdx.x] = total;
}

// One pass of a tile of 1024 kRounds keys: each goes behind all keys of smaller digits and behind those of its digit that
// come before. kCounted: sort_count has counted the tiles' digits; else every workgroup counts all keys, which takes
// less than a launch of its own up to kSortUncounted keys.
template <int kRounds, bool kCounted>
__global__ __launch_bounds__(kSortThreads) void sort_pass(SortArgs a) {
  __shared__ SortShared s;
  if ((int)blockIdx.x >= a.groups) return fill_rows(a.fill, blockIdx.x - a.groups, gridDim.x - a.groups);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, d = threadIdx.x;
  const int64_t first = (int64_t)blockIdx.x * (kRounds * kSortThreads);
  const uint32_t mask = (1u << a.bits) - 1;
  uint32_t key[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = first + (wave * kRounds + r) * 64 + lane;
    key[r] = i < a.count ? key_of(a, i) : ~0u;
  }
  if (!kCounted) {  // of the keys before the tile, and of the others, in the wavefronts' counters
    static_assert(kSortWaves == 2 * kCopies, "two sets of copies");
    for (int c = d; c < kSortWaves * kDigits; c += kSortThreads) (&s.count[0][0])[c] = 0;
    __syncthreads();
    for (int64_t i0 = 0; i0 < a.count; i0 += 8 * kSortThreads) {
      uint32_t digit[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t i = i0 + u * kSortThreads + threadIdx.x;
        digit[u] = i < a.count ? (key_of(a, i) >> a.shift) & mask : ~0u;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // whole numbers: any order
        const int set = i0 + u * kSortThreads + threadIdx.x < first ? 0 : kCopies;
        if (digit[u] != ~0u) atomicAdd(&s.count[set + d % kCopies][digit[u]], 1u);
      }
    }
    __syncthreads();
  }
  if (d < kDigits) {
    uint32_t total = 0, before = 0;
    if (kCounted) {
#pragma unroll 8
      for (int g = 0; g < a.groups; ++g) {
        const uint32_t c = a.counts[(int64_t)g * kDigits + d];
        if (g < (int)blockIdx.x) before += c;
        total += c;
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        before += s.count[c][d];
        total += s.count[kCopies + c][d];
      }
      total += before;
    }
    s.total[d] = total;
    s.before[d] = before;
  }
  __syncthreads();
  rank_keys<kRounds>(s, key, rank, a.shift, a.bits);
  place_digits(s, false);
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = first + (wave * kRounds + r) * 64 + lane;
    if (i >= a.count) continue;
    const uint32_t digit = (key[r] >> a.shift) & mask;
    const uint32_t to = s.base[digit] + s.count[wave][digit] + rank[r];
    a.keys_out[to] = key[r];
    a.from_out[to] = a.from ? a.from[i] : (uint32_t)i;
  }
}

// ---------------------------------------------------------------------------
// the gradient: sums
// ---------------------------------------------------------------------------

// A lane's V columns of a row, from p on: the sum rounded, on top of `old` where the caller accumulates. The first
// `skip` belong to the neighbour before (V: all of them).
template <bool kAccumulate, typename T, int V>
__device__ __forceinline__ void write_row(T* p, int skip, float scale, const float (&sum)[V], const T (&old)[V]) {
  if (skip == V) return;
  T o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = (T)(kAccumulate ? fmaf(sum[e], scale, (float)old[e]) : sum[e] * scale);
  if (skip == 0) {
    __builtin_memcpy(p, o, 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e >= skip) p[e] = o[e];
  }
}

// The same of a row shorter than a chunk, by lane 0.
template <typename T, int V>
__device__ __forceinline__ void write_narrow(const EmbeddingGradientArgs& a, uint32_t row, const float (&sum)[V]) {
  T* p = static_cast<T*>(a.dtable) + (int64_t)row * a.lddt;
  if ((threadIdx.x & 63) != 0) return;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < (int)a.k) p[e] = (T)(a.accumulate ? fmaf(sum[e], a.scale, (float)p[e]) : sum[e] * a.scale);
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

// kNarrow: rows shorter than a chunk, which lane 0 has alone. kAccumulate: what the table holds is loaded along with
// the tokens; loaded where a row ends, each of a piece's rows would wait for it (1777 tokens x 1111: 51 us).
template <typename T, bool kNarrow, bool kAccumulate>
__global__ __launch_bounds__(256) void embedding_sums(EmbeddingGradientArgs a, int64_t pieces, int64_t slabs) {
  constexpr int V = kChunkOf<T>;
  const int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= pieces * slabs) return;
  const int64_t piece = task / slabs, slab = task % slabs, s0 = piece * a.piece;
  const int lane = threadIdx.x & 63;
  const uint32_t none = (uint32_t)a.rows;
  // the first lanes: the piece; the next one: the token after; lane 63: the one before
  const int64_t i = lane == 63 ? s0 - 1 : s0 + (lane <= a.piece ? lane : a.piece);
  const uint32_t key = i >= 0 && i < a.count ? a.keys[0][i] : none;
  const uint32_t from = i >= 0 && i < a.count ? a.from[0][i] : 0;
  const int tokens = __popcll(__ballot(lane < a.piece && key < none));  // those without a row come last
  if (tokens == 0) return;
  int64_t at;
  int skip;
  lane_columns<V, kNarrow>(a.k, slab, &at, &skip);
  if (kNarrow && skip < V) skip = 0;
  const T* G = static_cast<const T*>(a.g) + at;
  float sum[V] = {};
  bool crosses = __builtin_amdgcn_readlane(key, 63) == __builtin_amdgcn_readlane(key, 0);  // the first row began earlier
  const bool on = tokens == a.piece;
  for (int j0 = 0; j0 < tokens; j0 += kSumBatch) {
    T x[kSumBatch][V], old[kSumBatch][V];
#pragma unroll
    for (int b = 0; b < kSumBatch; ++b) {
      const int j = j0 + b < tokens ? j0 + b : tokens - 1;
      if (kAccumulate && !kNarrow)
        __builtin_memcpy(old[b], static_cast<const T*>(a.dtable) + (int64_t)(uint32_t)__builtin_amdgcn_readlane(key, j) * a.lddt + at, 16);
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
        write_narrow<T, V>(a, row, sum);
      } else {
        write_row<kAccumulate, T, V>(static_cast<T*>(a.dtable) + (int64_t)row * a.lddt + at, skip, a.scale, sum, old[b]);
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
  const int64_t piece = blockIdx.x / slabs, slab = blockIdx.x % slabs, end = (piece + 1) * a.piece;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t none = (uint32_t)a.rows;
  const uint32_t* keys = a.keys[0];
  if (end >= a.count) return;
  const uint32_t key = keys[end - 1];
  if (key >= none || keys[end] != key) return;  // no row goes on
  const int64_t start = piece * a.piece;
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
    const int64_t next = (q0 + lane + 1) * a.piece;
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
  if (kNarrow) return write_narrow<T, V>(a, key, sum);
  int64_t at;
  int skip;
  lane_columns<V, kNarrow>(a.k, slab, &at, &skip);
  T* p = static_cast<T*>(a.dtable) + (int64_t)key * a.lddt + at;
  T old[V] = {};
  if (a.accumulate) {
    __builtin_memcpy(old, p, 16);
    write_row<true, T, V>(p, skip, a.scale, sum, old);
  } else {
    write_row<false, T, V>(p, skip, a.scale, sum, old);
  }
}

constexpr int64_t kL2Bytes = 32 << 20;  // of the eight XCDs

template <typename T>
void embedding_for(const EmbeddingArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  const int64_t chunks = (a.k + V - 1) / V;
  const auto grid = [&](int lanes) {
    const int64_t groups = (a.count * lanes + 255) / 256, most = (int64_t)1 << 22;
    return (unsigned)(groups < most ? groups : most);
  };
  const bool streamed = a.count * a.k * (int64_t)sizeof(T) > kL2Bytes;
  const auto run = [&](auto lanes) {
    constexpr int kLanes = decltype(lanes)::value;
    if (streamed) embedding_rows<T, kLanes, false, true><<<grid(kLanes), 256, 0, s>>>(a);
    else embedding_rows<T, kLanes, false, false><<<grid(kLanes), 256, 0, s>>>(a);
  };
  if (a.k < V) embedding_rows<T, 4, true, false><<<grid(4), 256, 0, s>>>(a);
  else if (chunks <= 32) run(std::integral_constant<int, 16>());
  else if (chunks <= 128) run(std::integral_constant<int, 64>());
  else run(std::integral_constant<int, 256>());
}

template <typename T>
void sums_for(const EmbeddingGradientArgs& a, hipStream_t s) {
  constexpr int V = kChunkOf<T>;
  const int64_t pieces = piece_count(a.count, a.piece), slabs = (a.k + 64 * V - 1) / (64 * V);
  const unsigned groups = (unsigned)((pieces * slabs + 3) / 4);
  const auto run = [&](auto narrow) {
    constexpr bool kNarrow = decltype(narrow)::value;
    if (a.accumulate) embedding_sums<T, kNarrow, true><<<groups, 256, 0, s>>>(a, pieces, slabs);
    else embedding_sums<T, kNarrow, false><<<groups, 256, 0, s>>>(a, pieces, slabs);
    if (pieces > 1) embedding_join<T, kNarrow><<<(unsigned)(pieces * slabs), 256, 0, s>>>(a, pieces, slabs);
  };
  if (a.k < V) run(std::true_type());
  else run(std::false_type());
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
  q.end_bit = bits;
  const bool alone = q.groups <= 1, counted = a.count > kSortUncounted;
  const int launches = alone ? 1 : counted ? 2 * passes : passes;
  const int fillers = a.accumulate ? 0 : 512;
  for (int l = 0; l < launches; ++l) {
    q.fill.first = a.accumulate ? 0 : a.rows * l / launches;
    q.fill.end = a.accumulate ? 0 : a.rows * (l + 1) / launches;
    const unsigned grid = (unsigned)(q.groups + fillers);
    if (grid == 0) return hipSuccess;
    const int pass = counted ? l / 2 : l, to = pass & 1;
    q.ids = pass == 0 ? a.ids : nullptr;
    q.keys = pass == 0 ? nullptr : a.keys[to ^ 1];
    q.from = pass == 0 ? nullptr : a.from[to ^ 1];
    q.keys_out = a.keys[to];
    q.from_out = a.from[to];
    q.shift = pass * q.bits;
    if (alone && a.count <= kSortThreads) sort_all<1><<<grid, kSortThreads, 0, s>>>(q);
    else if (alone && a.count <= 2 * kSortThreads) sort_all<2><<<grid, kSortThreads, 0, s>>>(q);
    else if (alone) sort_all<kSortAlone / kSortThreads><<<grid, kSortThreads, 0, s>>>(q);
    else if (!counted) sort_pass<1, false><<<grid, kSortThreads, 0, s>>>(q);
    else if (l % 2 == 0) sort_count<<<grid, kSortThreads, 0, s>>>(q);
    else sort_pass<kCountedTile / kSortThreads, true><<<grid, kSortThreads, 0, s>>>(q);
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
