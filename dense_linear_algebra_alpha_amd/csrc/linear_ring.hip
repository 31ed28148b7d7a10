// Products of matrices whose rows are 16-byte aligned: large tiles fed through a ring of LDS slots.
//
// A workgroup of four wavefronts (2 x 2) forms a BM x BN tile of C. The contraction advances in
// stages of 64 bytes of a row (32 steps of 16-bit elements, 16 of fp32). A stage's two operand tiles go
// from memory straight into an LDS slot (16-byte loads to LDS, no registers); the ring holds four
// slots. While the products of stage t run, the fragments of stage t + 1 are read from LDS into
// registers and stages t + 2 .. t + 4 are on their way, so a load has three stages (at 256 x 256 about
// 3000 cycles) to arrive. Stage t's slot is free as soon as every wavefront has passed the barrier at
// the start of stage t (its fragments were read during stage t - 1), and takes stage t + 4.
//
// Per stage and wavefront a BM x BN tile reads (BM + BN) / 2 * 64 bytes of LDS for BM / 2 * BN / 2 * 64
// operations: four wavefronts of 128 x 128 rather than eight of 128 x 64 keep LDS reads (128 bytes a
// cycle and CU) at half of the matrix unit's time.
//
// LDS layout. Contraction contiguous in memory: a slot's rows hold 4 chunks of 16 bytes; chunk c of
// row r lies at c ^ (r / 2 & 3), so that any 8 neighbouring rows that a fragment reads at one chunk
// cover 128 bytes of banks. Contraction strided in memory (the gradient's products): a slot's rows are
// the steps, in units of 16 neighbours of the kept index, permuted by the step (Operand::key); of
// 16-bit elements the transposing LDS read gives each lane 4 steps of its neighbour. The loads to
// LDS write lanes in order, so the permutations are applied to the addresses that they read.
#include "linear_util.h"

namespace xtvxy {
namespace {

constexpr int kThreads = 256;
constexpr int kRing = 4;     // LDS slots
constexpr uint32_t kNowhere = 0xfffffff0u;  // beyond any tile's extent: such a load returns zero

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_byte;

template <typename T>
struct Stage {
  static constexpr int kChunk = 16 / sizeof(T);     // elements of a 16-byte chunk
  static constexpr int kSteps = 4 * kChunk;         // contraction steps of a stage: 64 bytes of a row
  typedef typename Vec<T>::x8 frag;                 // a lane's share of a 16-row fragment
};
template <>
struct Stage<float> {
  static constexpr int kChunk = 4;
  static constexpr int kSteps = 16;
  typedef f32x4 frag;
};

// One operand's tile of R rows of the kept index and one stage of the contraction: its loads into an
// LDS slot (R * 64 bytes, R / 16 loads of 1 KiB, R / 64 of them by each wavefront) and its fragments.
template <typename T, int R, bool kMajor>
struct Operand {
  static constexpr int kLoads = R / 64;
  static constexpr int kBytes = R * 64;
  static constexpr int kSize = sizeof(T), kChunk = Stage<T>::kChunk, kSteps = Stage<T>::kSteps;
  typedef typename Stage<T>::frag frag;

  const char* base;        // of the next stage to load: its first step, the tile's first row
  int64_t stage_bytes;     // from one stage to the next
  int64_t outer_bytes;     // of rows (steps) before the last one of the tile (a step)
  int32_t inner;           // rows of the tile that exist, in whole chunks (steps strided)
  uint32_t offset[kLoads]; // of this lane, per load, from base
  int32_t lane_step;       // first contraction step of this lane's chunk (steps contiguous)

  // The units that a step's row is permuted in: 32 bytes (16-bit, read 4 steps at a time by a group
  // of 16 lanes) or 64 bytes (fp32, read a step at a time).
  static __device__ __forceinline__ int key(int k) {
    if (kSize == 4) return (k >> 2) & 3 & (R / 16 - 1);
    return ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
  }

  // rows: of the kept index from the tile's first on; k0: the first step.
  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (!kMajor) {
      base = static_cast<const char*>(p) + (r0 * ld + k0) * kSize;
      stage_bytes = kSteps * kSize;
      outer_bytes = ((rows < R ? rows : R) - 1) * ld * kSize;
      const int chunk = (lane & 3) ^ ((lane >> 3) & 3);
      lane_step = chunk * kChunk;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        offset[j] = (uint32_t)(((wave * kLoads + j) * 16 + (lane >> 2)) * ld * kSize) + chunk * 16;
    } else {
      base = static_cast<const char*>(p) + (k0 * ld + r0) * kSize;
      stage_bytes = kSteps * ld * kSize;
      outer_bytes = ld * kSize;
      inner = ((int32_t)(rows < R ? rows : R) + kChunk - 1) / kChunk * kChunk;
      constexpr int kChunks = R / kChunk;            // of a step's row
      constexpr int kUnit = kSize == 4 ? 4 : 2;      // chunks of a unit
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int at = (wave * kLoads + j) * 64 + lane, k = at / kChunks, slot = at % kChunks;
        const int chunk = slot ^ (key(k) * kUnit);
        offset[j] = chunk * kChunk < inner ? (uint32_t)(k * ld * kSize) + chunk * 16 : kNowhere;
      }
    }
  }

  // The buffer descriptor of the next stage, of which `left` contraction steps exist.
  __device__ __forceinline__ u32x4 next(int32_t left) {
    // bytes from base to the end of what the stage may read: beyond them a load returns zero. In
    // whole chunks: of a word that straddles the end nothing would be read.
    const int32_t steps = left < kSteps ? left : kSteps;
    uint32_t extent = 0;
    if (left > 0)
      extent = kMajor ? (uint32_t)(steps - 1) * (uint32_t)outer_bytes + (uint32_t)inner * kSize
                      : (uint32_t)outer_bytes + (uint32_t)((steps + kChunk - 1) / kChunk * kChunk) * kSize;
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    base += stage_bytes;
    return u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, extent, 0x00027000u};
  }

  // Load j of a stage of which `left` steps exist, into the slot at `lds`. Written out because the
  // compiler makes transposing LDS reads wait for every load to LDS that it knows of; it has no
  // result register, and the kernel's own waits and barriers order it with the reads of its slot.
  __device__ __forceinline__ void load(u32x4 rsrc, uint32_t lds, int j, int32_t left) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t o = offset[j];
    if (!kMajor) o = lane_step < left ? o : kNowhere;  // the rest of a memory row is the next row's
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds + (wave * kLoads + j) * 1024), "v"(o), "s"(rsrc)
                 : "memory");  // m0 is written next to each use, by the compiler as well
  }

  // This lane's byte offset in a slot for the fragments of a wavefront's rows, from w on.
  static __device__ __forceinline__ uint32_t fragment_base(int w) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    if (!kMajor) return (w + r) * 64 + ((g ^ ((r >> 1) & 3)) << 4);
    if (kSize == 4) return g * 4 * R * 4 + (((w >> 4) ^ key(g * 4)) << 6) + r * 4;
    const int k = g * 8 + (r >> 2);
    return k * R * 2 + (((w >> 4) ^ key(k)) << 5) + (r & 3) * 8;
  }

  // Fragment f: rows w + 16 f + 0..15, the stage's steps; lane group g has steps g kSteps / 4 on.
  static __device__ __forceinline__ frag fragment(lds_byte* slot, uint32_t at, int f) {
    if (!kMajor) return *(__attribute__((address_space(3))) frag*)(slot + at + f * 1024);
    if constexpr (kSize == 4) {
      lds_byte* p = slot + (at ^ (uint32_t)(f << 6));
      frag v;
#pragma unroll
      for (int s = 0; s < 4; ++s) v[s] = *(__attribute__((address_space(3))) float*)(p + s * R * 4);
      return v;
    } else {
      lds_byte* p = slot + (at ^ (uint32_t)(f << 5));
      union {
        s16x4 half[2];
        frag all;
      } u;
      u.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
      u.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p + 4 * R * 2));
      return u.all;
    }
  }
};

// acc += the product of two fragments, in place. Written out because the compiler otherwise moves the
// 256 sums of a 256 x 256 tile between registers (3 moves per product); the sums' first reader after
// the loop waits for the last product itself.
__device__ __forceinline__ void mfma_in_place(f32x4& acc, bf16x8 a, bf16x8 b, int) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_in_place(f32x4& acc, f16x8 a, f16x8 b, int) {
  asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// fp32: one step of each lane group, the s-th of its four
__device__ __forceinline__ void mfma_in_place(f32x4& acc, f32x4 a, f32x4 b, int s) {
  asm volatile("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+a"(acc) : "v"(a[s]), "v"(b[s]));
}

// The s_waitcnt operand that waits until at most `vm` memory and `lgkm` LDS operations are under way.
constexpr int waitcnt(int vm, int lgkm) { return (vm & 15) | (7 << 4) | (lgkm << 8) | ((vm >> 4) << 14); }

// Tile of a workgroup: workgroups go to the 8 XCDs in turn, each of which has an L2 of its own, so
// each XCD takes a contiguous range of the tiles, ordered in bands of kBand tile rows.
__device__ __forceinline__ void tile_of(uint32_t id, int64_t tiles_m, int64_t tiles_n, int64_t* tm, int64_t* tn) {
  constexpr int kXcds = 8, kBand = 4;
  const uint32_t tiles = (uint32_t)(tiles_m * tiles_n);
  const uint32_t x = id % kXcds, q = tiles / kXcds, r = tiles % kXcds;
  const uint32_t t = x * q + (x < r ? x : r) + id / kXcds;
  const uint32_t band_tiles = kBand * (uint32_t)tiles_n, band = t / band_tiles, in = t % band_tiles;
  const uint32_t rows = (uint32_t)tiles_m - band * kBand < kBand ? (uint32_t)tiles_m - band * kBand : kBand;
  *tm = band * kBand + in % rows;
  *tn = in / rows;
}

// Where the four columns from 4 c on of a staged row lie (in floats): the rows' pitch is a multiple of
// the banks, so the chunks are permuted by the row.
template <int WN>
__device__ __forceinline__ int staged_at(int row, int c) {
  return row * WN + ((c ^ (row & 7)) << 2);
}

template <int WN>
__device__ __forceinline__ f32x8 staged8(const float* area, int row, int c8) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(area + staged_at<WN>(row, 2 * c8));
  const f32x4 hi = *reinterpret_cast<const f32x4*>(area + staged_at<WN>(row, 2 * c8 + 1));
  return {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// The epilogue of a wavefront's staged rows from (i0, j0) on, 8 columns a lane.
template <typename T, int kAct, int WN, int kRows>
__device__ __forceinline__ void epilogue_rows(const float* area, const ProductArgs& a, int64_t i0, int64_t j0) {
  typedef typename Vec<T>::x8 v8;
  constexpr int kLanes = WN / 8, kStep = 64 / kLanes;  // lanes of a row, rows at once
  const LinearEpilogue& e = a.e;
  const int lane = threadIdx.x & 63, c8 = lane % kLanes;
  const int64_t j = j0 + c8 * 8;
  const int count = a.n - j >= 8 ? 8 : (a.n > j ? (int)(a.n - j) : 0);
  if (count == 0) return;
  const bool wide = e.wide8 && count == 8;
  f32x8 bias = {};
  if (e.bias)
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < count) bias[c] = e.bias[j + c];
  const int rows = a.m - i0 >= kRows ? kRows : (int)(a.m - i0);
  if (wide) {
    const T* res = static_cast<const T*>(e.residual) + (e.residual ? i0 * e.ldr + j : 0);
    T* pre = static_cast<T*>(e.pre) + (e.pre ? i0 * e.ldp + j : 0);
    T* out = static_cast<T*>(e.out) + i0 * e.ldo + j;
#pragma unroll 4
    for (int row = lane / kLanes; row < rows; row += kStep) {
      v8 rv = {};
      if (e.residual) rv = *reinterpret_cast<const v8*>(res + row * e.ldr);
      f32x8 z = staged8<WN>(area, row, c8) + bias;
      v8 o;
      if (e.pre) {
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = (T)z[c];
        *reinterpret_cast<v8*>(pre + row * e.ldp) = o;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        float y = activation<sizeof(T) == 2, kAct>(z[c]);
        if (e.residual) y += (float)rv[c];
        o[c] = (T)y;
      }
      *reinterpret_cast<v8*>(out + row * e.ldo) = o;
    }
  } else {
    for (int row = lane / kLanes; row < rows; row += kStep) {
      const f32x8 z = staged8<WN>(area, row, c8) + bias;
      const int64_t i = i0 + row;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c >= count) break;
        if (e.pre) static_cast<T*>(e.pre)[i * e.ldp + j + c] = (T)z[c];
        float y = activation<sizeof(T) == 2, kAct>(z[c]);
        if (e.residual) y += (float)static_cast<const T*>(e.residual)[i * e.ldr + j + c];
        static_cast<T*>(e.out)[i * e.ldo + j + c] = (T)y;
      }
    }
  }
}

template <typename T, int WN, int kRows>
__device__ __forceinline__ void epilogue_any(const float* area, const ProductArgs& a, int64_t i0, int64_t j0) {
  switch (a.e.act) {
    case XTVXY_ACT_RELU: epilogue_rows<T, XTVXY_ACT_RELU, WN, kRows>(area, a, i0, j0); break;
    case XTVXY_ACT_GELU: epilogue_rows<T, XTVXY_ACT_GELU, WN, kRows>(area, a, i0, j0); break;
    case XTVXY_ACT_GELU_TANH: epilogue_rows<T, XTVXY_ACT_GELU_TANH, WN, kRows>(area, a, i0, j0); break;
    case XTVXY_ACT_SILU: epilogue_rows<T, XTVXY_ACT_SILU, WN, kRows>(area, a, i0, j0); break;
    default: epilogue_rows<T, XTVXY_ACT_NONE, WN, kRows>(area, a, i0, j0); break;
  }
}

// The staged rows as one part of a split product.
template <int WN, int kRows>
__device__ __forceinline__ void partial_rows(const float* area, const ProductArgs& a, uint32_t split, int64_t i0, int64_t j0) {
  constexpr int kLanes = WN / 4, kStep = 64 / kLanes;
  const int lane = threadIdx.x & 63, c4 = lane % kLanes;
  const int64_t j = j0 + c4 * 4;
  if (j >= a.n) return;
  const int count = a.n - j >= 4 ? 4 : (int)(a.n - j);
  const int rows = a.m - i0 >= kRows ? kRows : (int)(a.m - i0);
  float* p = a.partial + ((int64_t)split * a.m + i0) * a.n + j;
  for (int row = lane / kLanes; row < rows; row += kStep)
    store4<float>(p + row * a.n, *reinterpret_cast<const f32x4*>(area + staged_at<WN>(row, c4)), count, a.n % 4 == 0);
}

// Workgroup `id` of a product's tiles x splits, with `ring` of 4 (BM + BN) 64 bytes of LDS.
template <typename T, int BM, int BN, bool kAMajor, bool kBMajor>
__device__ __forceinline__ void ring_tile(const ProductArgs& a, uint32_t id, uint8_t* ring) {
  typedef typename Stage<T>::frag frag;
  typedef Operand<T, BM, kAMajor> OpA;
  typedef Operand<T, BN, kBMajor> OpB;
  constexpr int kStage = Stage<T>::kSteps;
  constexpr int kSlot = OpA::kBytes + OpB::kBytes;
  constexpr int FA = BM / 32, FB = BN / 32;  // fragments of a wavefront's BM / 2 x BN / 2
  constexpr int kLoads = OpA::kLoads + OpB::kLoads;
  lds_byte* lds = (lds_byte*)ring;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);

  const int64_t tiles_m = (a.m + BM - 1) / BM, tiles_n = (a.n + BN - 1) / BN;
  const uint32_t tiles = (uint32_t)(tiles_m * tiles_n), split = id / tiles;
  int64_t tm, tn;
  tile_of(id % tiles, tiles_m, tiles_n, &tm, &tn);
  const int64_t i0 = tm * BM, j0 = tn * BN;
  const int64_t k0 = (int64_t)split * a.k_per_split;
  const int64_t k_end = k0 + a.k_per_split < a.k ? k0 + a.k_per_split : a.k;
  int32_t left = (int32_t)(k_end - k0);
  const int32_t stages = (left + kStage - 1) / kStage;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = (wave >> 1) * (BM / 2), wj = (wave & 1) * (BN / 2);

  OpA oa;
  OpB ob;
  oa.init(a.A, a.lda, i0, a.m - i0, k0);
  ob.init(a.B, a.ldb, j0, a.n - j0, k0);
  const uint32_t at_a = OpA::fragment_base(wi), at_b = OpB::fragment_base(wj);
  f32x4 acc[FA][FB] = {};
  frag fa[2][FA], fb[2][FB];

#pragma unroll
  for (int s = 0; s < kRing; ++s) {
    const u32x4 ra = oa.next(left), rb = ob.next(left);
#pragma unroll
    for (int j = 0; j < OpA::kLoads; ++j) oa.load(ra, lds0 + s * kSlot, j, left);
#pragma unroll
    for (int j = 0; j < OpB::kLoads; ++j) ob.load(rb, lds0 + s * kSlot + OpA::kBytes, j, left);
    left -= kStage;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(waitcnt(3 * kLoads, 15));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int f = 0; f < FA; ++f) fa[0][f] = OpA::fragment(lds, at_a, f);
#pragma unroll
  for (int f = 0; f < FB; ++f) fb[0][f] = OpB::fragment(lds + OpA::kBytes, at_b, f);

  auto stage = [&](int now, uint32_t slot) {
    // stage t + 1 has arrived (two younger ones may be on their way), and every wavefront has stage t's
    // fragments in registers
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt(2 * kLoads, 0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint32_t here = lds0 + slot * kSlot;
    lds_byte* next = lds + ((slot + 1) & (kRing - 1)) * kSlot;
    const u32x4 ra = oa.next(left), rb = ob.next(left);
    // The loads of stage t + 4 and the fragments of stage t + 1 are issued between the products, a few
    // at a time: the matrix unit is never left waiting behind a queue of them. (Past the last stage the
    // fragments are zeros or leftovers of the ring that nothing uses.)
    constexpr int kGroups = FA + FB, kProducts = FA * FB * (sizeof(T) == 4 ? 4 : 1);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if ((q + 1) * kLoads / kGroups > q * kLoads / kGroups) {
        const int j = q * kLoads / kGroups;
        if (j < OpA::kLoads) oa.load(ra, here, j, left);
        else ob.load(rb, here + OpA::kBytes, j - OpA::kLoads, left);
      }
      if (q < FA) fa[now ^ 1][q] = OpA::fragment(next, at_a, q);
      else fb[now ^ 1][q - FA] = OpB::fragment(next + OpA::kBytes, at_b, q - FA);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = q * kProducts / kGroups; c < (q + 1) * kProducts / kGroups; ++c)
        mfma_in_place(acc[c / FB % FA][c % FB], fb[now][c % FB], fa[now][c / FB % FA], c / (FA * FB));
      __builtin_amdgcn_sched_barrier(0);
    }
    left -= kStage;
  };
  // stages in pairs, so that the two sets of fragments keep their registers; where their number is odd
  // the last one's loads all lie beyond the extent and its products add zeros
  for (int32_t t = 0; t < stages; t += 2) {
    stage(0, t & (kRing - 1));
    stage(1, (t + 1) & (kRing - 1));
  }
  // no load to LDS outlives the workgroup, and the last products are through before their sums are read
  asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int c = 0; c < FA * FB; ++c) asm volatile("" : "+a"(acc[c / FB][c % FB]));

  __syncthreads();  // the ring is free: nobody reads fragments any more

  // The sums go through LDS, up to 64 rows of a wavefront at a time, so that a lane then has 8 neighbouring
  // columns and a row's lanes its whole width: 16-byte accesses of out, pre and residual.
  constexpr int WN = BN / 2, kRows = BM / 2 < 64 ? BM / 2 : 64;
  constexpr int kArea = kRows * WN * 4;  // bytes of a wavefront
  static_assert(4 * kArea <= kRing * kSlot, "the staged sums fit the ring");
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  float* area = reinterpret_cast<float*>(ring + wave * kArea);
#pragma unroll
  for (int part = 0; part < BM / 2 / kRows; ++part) {
#pragma unroll
    for (int x = 0; x < kRows / 16; ++x)
#pragma unroll
      for (int y = 0; y < FB; ++y)
        *reinterpret_cast<f32x4*>(area + staged_at<WN>(x * 16 + r, y * 4 + g)) = acc[part * (kRows / 16) + x][y];
    __builtin_amdgcn_wave_barrier();
    const int64_t i = i0 + wi + part * kRows, j = j0 + wj;
    if (a.splits > 1)
      partial_rows<WN, kRows>(area, a, split, i, j);
    else
      epilogue_any<T, WN, kRows>(area, a, i, j);
    __builtin_amdgcn_wave_barrier();
  }
}

constexpr int ring_bytes(int tile) { return kRing * 2 * tile * 64; }

template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void layer_ring(ProductArgs a) {
  __shared__ __align__(1024) uint8_t ring[ring_bytes(TILE)];
  ring_tile<T, TILE, TILE, false, false>(a, blockIdx.x, ring);
}

// The gradient's two products in one launch (the second's workgroups fill the CUs that the first's last
// round leaves), and the sum of the row groups' column sums.
template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, TILE > 128 ? 1 : 2) void gradient_ring(GradientArgs a) {
  __shared__ __align__(1024) uint8_t ring[ring_bytes(TILE)];
  uint32_t id = blockIdx.x;
  if (id < a.dx_groups) return ring_tile<T, TILE, TILE, false, true>(a.dx, id, ring);
  id -= a.dx_groups;
  if (id < a.dw_groups) return ring_tile<T, TILE, TILE, true, true>(a.dw, id, ring);
  column_sum(a.sums, a.sum_rows, a.n, a.db, id - a.dw_groups, reinterpret_cast<double*>(ring));
}

uint32_t groups_of(const ProductArgs& a, int tile) {
  return (uint32_t)(((a.m + tile - 1) / tile) * ((a.n + tile - 1) / tile) * a.splits);
}

template <typename T, int TILE>
hipError_t layer_for(const ProductArgs& a, hipStream_t s) {
  layer_ring<T, TILE><<<groups_of(a, TILE), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int TILE>
hipError_t gradient_for(GradientArgs a, hipStream_t s) {
  a.dx_groups = a.dx.m > 0 ? groups_of(a.dx, TILE) : 0;
  a.dw_groups = a.dw.m > 0 ? groups_of(a.dw, TILE) : 0;
  const uint32_t columns = a.db ? (uint32_t)((a.n + kSumColumns - 1) / kSumColumns) : 0;
  if (a.dx_groups + a.dw_groups + columns == 0) return hipSuccess;
  gradient_ring<T, TILE><<<a.dx_groups + a.dw_groups + columns, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t layer_type(const ProductArgs& a, int tile, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (tile == 256) return layer_for<T, 256>(a, s);
  }
  if (tile == 128) return layer_for<T, 128>(a, s);
  return layer_for<T, 64>(a, s);
}

template <typename T>
hipError_t gradient_type(const GradientArgs& a, int tile, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (tile == 256) return gradient_for<T, 256>(a, s);
  }
  if (tile == 128) return gradient_for<T, 128>(a, s);
  return gradient_for<T, 64>(a, s);
}

}  // namespace

hipError_t launch_layer_ring(const ProductArgs& a, int tile, hipStream_t s) {
  if (a.type == kBf16) return layer_type<__bf16>(a, tile, s);
  if (a.type == kF16) return layer_type<_Float16>(a, tile, s);
  return layer_type<float>(a, tile, s);
}

hipError_t launch_gradient_ring(const GradientArgs& a, int type, int tile, hipStream_t s) {
  if (type == kBf16) return gradient_type<__bf16>(a, tile, s);
  if (type == kF16) return gradient_type<_Float16>(a, tile, s);
  return gradient_type<float>(a, tile, s);
}

}  // namespace xtvxy
