// Products of matrices whose rows are 16-byte aligned: large tiles fed through a ring of LDS slots.
//
// C(i, j) = sum over k of A(i, k) B(j, k). A workgroup of four wavefronts (2 x 2) forms a BM x BN tile of C;
// the sums stay in registers (256 of a lane for 256 x 256). The contraction advances in stages: two operand
// tiles of 64 bytes of a row (32 steps of 16-bit elements, 16 of fp32), or of 128 bytes for 256 x 256, go
// from memory straight into an LDS slot (16-byte loads to LDS, no registers). While the products of a
// stage run, the next fragments are read from LDS into registers and later stages are on their way.
//
// What bounds it. 8192^3 in bf16 takes 720 to 850 us (1.5 to 1.3 PFLOP/s: the clock falls as the card warms; the
// library's product 660 to 850 on the same cards): the power. From call to call the clock fell from 2.00 to 1.65
// GHz while the matrix unit went from 63 to 72% busy, 1.2 busy cycles a nanosecond and SIMD throughout. Per
// 64 bytes and wavefront a BM x BN tile reads (BM + BN) / 2 * 64 bytes of LDS for BM / 2 * BN / 2 * 64 operations:
// four wavefronts of 128 x 128 rather than eight of 128 x 64 keep LDS reads (128 bytes a cycle and CU) at half
// of the matrix unit's time; 128 x 128 tiles take all of it (0.27 us a stage where a quarter of 256 x 256's is
// 0.18), and 256 x 128 ones, one on a CU, lost to both on 44 of 46 shapes. fp32 4096 x 1024 x 1024 takes 65 to 77 us
// (131 to 112 TFLOP/s; 154 is what the library reaches at 8192^3).
//
// LDS layout. Contraction contiguous in memory: a slot's rows hold 4 chunks of 16 bytes; chunk c of
// row r lies at c ^ (r / 2 & 3), so that any 8 neighbouring rows that a fragment reads at one chunk
// cover 128 bytes of banks. Contraction strided in memory (the gradient's products): a slot's rows are
// the steps, in units of 16 neighbours of the kept index, permuted by the step (Operand::key); of
// 16-bit elements the transposing LDS read gives each lane 4 steps of its neighbour. The loads to
// LDS write lanes in order, so the permutations are applied to the addresses that they read.
#pragma once

#include "linear_util.h"

namespace xtvxy {
namespace {

constexpr int kThreads = 256;
constexpr int kRing = 4;     // LDS slots (eight gain nothing, not even for a lone 64 x 64 workgroup)
constexpr uint32_t kNowhere = 0xc0000000u;  // beyond any tile's extent: such a load returns zero
// Four loads share a setting of their LDS address: an instruction's own offset (up to 4095) counts for
// memory and LDS alike. Descriptors begin this far before their data, so that taking those offsets from
// the lanes' ones leaves none negative.
constexpr uint32_t kBefore = 4096;

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
template <typename T, int R, bool kMajor, int H>
struct Operand {
  static constexpr int kLoads = R / 64 * H;
  static constexpr int kBytes = R * 64 * H;
  static constexpr int kSize = sizeof(T), kChunk = Stage<T>::kChunk, kSteps = Stage<T>::kSteps * H;
  typedef typename Stage<T>::frag frag;

  u32x4 rsrc;              // buffer descriptor of the next stage to load: its first step, the tile's first
                           // row, kBefore bytes earlier, and the bytes that a whole stage may read
  int64_t stage_bytes;     // from one stage to the next
  uint32_t outer_bytes;    // of rows (steps) before the last one of the tile (a step)
  int32_t inner;           // rows of the tile that exist, in whole chunks (steps strided)
  uint32_t offset[kLoads]; // of this lane, per load
  int32_t lane_step;       // first contraction step of this lane's chunk (steps contiguous)

  // The units that a step's row is permuted in: 32 bytes (16-bit, read 4 steps at a time by a group
  // of 16 lanes) or 64 bytes (fp32, read a step at a time).
  static __device__ __forceinline__ int key(int k) {
    if (kSize == 4) return (k >> 2) & 3 & (R / 16 - 1);
    return ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
  }

  // What a row's chunks are permuted by (contraction contiguous).
  static __device__ __forceinline__ int row_key(int row) { return H == 2 ? row & 7 : (row >> 1) & 3; }

  // rows: of the kept index from the tile's first on; k0: the first step.
  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const char* base;
    if (!kMajor) {
      base = static_cast<const char*>(p) + (r0 * ld + k0) * kSize;
      stage_bytes = kSteps * kSize;
      outer_bytes = (uint32_t)(((rows < R ? rows : R) - 1) * ld * kSize);
      constexpr int kRow = 4 * H;  // chunks of a row
      const int row = lane / kRow, chunk = (lane % kRow) ^ row_key(row);
      lane_step = chunk * kChunk;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        offset[j] = (uint32_t)(((wave * kLoads + j) * (64 / kRow) + row) * ld * kSize) + chunk * 16;
    } else {
      base = static_cast<const char*>(p) + (k0 * ld + r0) * kSize;
      stage_bytes = kSteps * ld * kSize;
      outer_bytes = (uint32_t)(ld * kSize);
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
#pragma unroll
    for (int j = 0; j < kLoads; ++j) offset[j] += kBefore - (j & 3) * 1024;
    const uint64_t at = reinterpret_cast<uint64_t>(base) - kBefore;
    rsrc = u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, extent(kSteps), 0x00027000u};
  }

  // Bytes from the descriptor's start to the end of what a stage of `steps` may read: beyond them a load
  // returns zero. In whole chunks: of a word that straddles the end nothing would be read.
  __device__ __forceinline__ uint32_t extent(int32_t steps) const {
    if (steps <= 0) return 0;
    return kBefore + (kMajor ? (uint32_t)(steps - 1) * outer_bytes + (uint32_t)inner * kSize
                             : outer_bytes + (uint32_t)((steps + kChunk - 1) / kChunk * kChunk) * kSize);
  }

  // Called before the loads of a stage of which only `left` < kSteps steps exist (none from there on).
  __device__ __forceinline__ void tail(int32_t left) {
    rsrc[2] = extent(left);
    asm volatile("");  // a branch: selecting every lane's offset in every stage would cost as much as 4 products
    if (!kMajor) {  // the rest of a memory row is the next row's
#pragma unroll
      for (int j = 0; j < kLoads; ++j) offset[j] = lane_step < left ? offset[j] : kNowhere;
    }
  }

  // After the loads of a stage.
  __device__ __forceinline__ void advance() {
    const uint64_t at = ((uint64_t)rsrc[1] << 32 | rsrc[0]) + (uint64_t)stage_bytes;
    rsrc[0] = (uint32_t)at;
    rsrc[1] = (uint32_t)(at >> 32);
  }

  // Where this wavefront's loads j .. j + 3 (j a multiple of 4) go in the slot at `lds`; then load j.
  // Written out because the compiler makes transposing LDS reads wait for every load to LDS that it
  // knows of. A load has no result register, and the kernel's own waits and barriers order it with the
  // reads of its slot. m0 has no other use in these kernels; one instruction has to lie between its
  // setting and the load.
  static __device__ __forceinline__ void aim(uint32_t lds, int j) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    asm volatile("s_mov_b32 m0, %0" : : "s"(lds + (wave * kLoads + j) * 1024) : "memory");
  }
  __device__ __forceinline__ void load(int j) const {
    switch (j & 3) {
      case 0: asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(offset[j]), "s"(rsrc) : "memory"); break;
      case 1: asm volatile("buffer_load_dwordx4 %0, %1, 0 offen offset:1024 lds" : : "v"(offset[j]), "s"(rsrc) : "memory"); break;
      case 2: asm volatile("buffer_load_dwordx4 %0, %1, 0 offen offset:2048 lds" : : "v"(offset[j]), "s"(rsrc) : "memory"); break;
      default: asm volatile("buffer_load_dwordx4 %0, %1, 0 offen offset:3072 lds" : : "v"(offset[j]), "s"(rsrc) : "memory"); break;
    }
  }
  // All loads of a stage of which `left` steps exist.
  __device__ __forceinline__ void load_stage(uint32_t lds, int32_t left) {
    if (left < kSteps) tail(left);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if ((j & 3) == 0) {
        aim(lds, j);
        asm volatile("s_nop 0");
      }
      load(j);
    }
    advance();
  }

  // This lane's byte offset in a slot for the fragments of a wavefront's rows, from w on.
  static __device__ __forceinline__ uint32_t fragment_base(int w) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    if (!kMajor) return (w + r) * 64 * H + ((g ^ row_key(r)) << 4);
    if (kSize == 4) return g * 4 * R * 4 + (((w >> 4) ^ key(g * 4)) << 6) + r * 4;
    const int k = g * 8 + (r >> 2);
    return k * R * 2 + (((w >> 4) ^ key(k)) << 5) + (r & 3) * 8;
  }

  // Fragment f: rows w + 16 f + 0..15, half h of the stage's steps; lane group g has a quarter of them.
  static __device__ __forceinline__ frag fragment(lds_byte* slot, uint32_t at, int f, int h = 0) {
    if (!kMajor) return *(__attribute__((address_space(3))) frag*)(slot + (at ^ (uint32_t)(h * 64)) + f * 1024 * H);
    slot += h * (kSteps / H) * R * kSize;
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

// The staged rows as one part of a split tile: row-major in the tile's own area.
template <int WN, int kRows, int BN>
__device__ __forceinline__ void partial_rows(const float* area, float* p) {
  constexpr int kLanes = WN / 4, kStep = 64 / kLanes;
  const int lane = threadIdx.x & 63, c4 = lane % kLanes;
#pragma unroll 4
  for (int row = lane / kLanes; row < kRows; row += kStep)
    *reinterpret_cast<f32x4*>(p + row * BN + c4 * 4) = *reinterpret_cast<const f32x4*>(area + staged_at<WN>(row, c4));
}

// A wavefront's sums in registers: 16 x 16 tiles of the matrix instruction. stage() writes
// the part-th strip of `rows` rows to the wavefront's staging area.
template <int FA, int FB>
struct Sums16 {
  f32x4 acc[FA][FB];
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int c = 0; c < FA * FB; ++c) asm volatile("" : "+a"(acc[c / FB][c % FB]));
  }
  template <int WN>
  __device__ __forceinline__ void stage(float* area, int part, int rows) const {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int x = 0; x < FA; ++x)
#pragma unroll
      for (int y = 0; y < FB; ++y)
        if (x * 16 / rows == part)
          *reinterpret_cast<f32x4*>(area + staged_at<WN>(x * 16 % rows + r, y * 4 + g)) = acc[x][y];
  }
};
// A tile's place in its product.
struct TilePlace {
  float* part;  // where its sums go if it is one part of a split tile, else null
  int64_t i0, j0, k0;
  int32_t steps;
};
template <int BM, int BN>
__device__ __forceinline__ TilePlace place_of(const ProductArgs& a, uint32_t id) {
  TilePlace p;
  int64_t tm, tn, k_end = a.k;
  const uint32_t whole = (uint32_t)a.whole;
  p.part = nullptr;
  p.k0 = 0;
  if (id < whole) {
    tile_of(a, spread(id, whole), &tm, &tn);
  } else {
    const uint32_t rest = (uint32_t)a.tiles() - whole, split = (id - whole) / rest, r = (id - whole) % rest;
    tile_of(a, whole + spread(r, rest), &tm, &tn);
    if (a.splits > 1 || a.in_parts) p.part = a.partial + ((int64_t)split * rest + r) * (BM * BN);
    p.k0 = (int64_t)split * a.k_per_split;
    k_end = p.k0 + a.k_per_split < a.k ? p.k0 + a.k_per_split : a.k;
  }
  p.i0 = tm * BM;
  p.j0 = tn * BN;
  p.steps = (int32_t)(k_end - p.k0);
  return p;
}

// After the last stage, before the sums are read.
template <typename S>
__device__ __forceinline__ void end_of_products(S& sums) {
  // no load to LDS outlives the workgroup, and the last products are through before their sums are read
  asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
  sums.settle();
  __syncthreads();  // the ring is free: nobody reads fragments any more
}

// The sums go through LDS, up to 64 rows of a wavefront at a time, so that a lane then has 8 neighbouring
// columns and a row's lanes its whole width: 16-byte accesses of what is read and written.
template <int BM, int BN>
struct Strips {
  static constexpr int kWidth = BN / 2, kRows = BM / 2 < 64 ? BM / 2 : 64;
  static constexpr int kArea = kRows * kWidth * 4;  // bytes of a wavefront
  static_assert(4 * kArea <= kRing * (BM + BN) * 64, "the staged sums fit the ring");
};

// Issue op(0) .. op(ops - 1) between product(0) .. product(products - 1), spread evenly. With one
// wavefront on a SIMD the matrix unit runs dry where more than about three other instructions stand
// between two products (16 cycles at a 4-cycle issue), so they are pinned one by one.
template <int kOps, int kProducts, typename Op, typename Product>
__device__ __forceinline__ void interleave(Op op, Product product) {
#pragma unroll
  for (int c = 0; c < kProducts; ++c) {
    product(c);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = (c * kOps + kProducts - 1) / kProducts; i * kProducts < (c + 1) * kOps; ++i) {
      op(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The loads of a stage as a list of instructions: per four loads one setting of their LDS address.
template <typename OpA, typename OpB>
struct StageLoads {
  static constexpr int kA = OpA::kLoads + (OpA::kLoads + 3) / 4, kB = OpB::kLoads + (OpB::kLoads + 3) / 4;
  static constexpr int kOps = kA + kB;
  static __device__ __forceinline__ void issue(const OpA& oa, const OpB& ob, uint32_t lds, int i) {
    if (i < kA) {
      if (i % 5 == 0) OpA::aim(lds, i / 5 * 4);
      else oa.load(i / 5 * 4 + i % 5 - 1);
    } else {
      i -= kA;
      if (i % 5 == 0) OpB::aim(lds + OpA::kBytes, i / 5 * 4);
      else ob.load(i / 5 * 4 + i % 5 - 1);
    }
  }
};

// Workgroup `id` of a product's tiles x splits for 256 x 256 tiles of 16-bit elements. `end` finishes the tile. Stages of two
// halves (128 bytes of a row): a load takes whole 128-byte lines where the contraction is contiguous,
// which halves the requests to L2 against 64-byte stages, and there is one barrier per two halves. Two
// slots; stage t's slot is free once its second half's fragments are in registers, at the barrier in
// the middle of stage t, and takes stage t + 2, which has until the middle of stage t + 1 to arrive.
template <typename T, int BM, int BN, bool kAMajor, bool kBMajor, typename End>
__device__ __forceinline__ void ring_tile_halves(const ProductArgs& a, uint32_t id, uint8_t* ring, const End& end) {
  typedef typename Stage<T>::frag frag;
  typedef Operand<T, BM, kAMajor, 2> OpA;
  typedef Operand<T, BN, kBMajor, 2> OpB;
  typedef StageLoads<OpA, OpB> Loads;
  constexpr int kStage = OpA::kSteps, kSlot = OpA::kBytes + OpB::kBytes;
  constexpr int FA = BM / 32, FB = BN / 32, kProducts = FA * FB, kReads = FA + FB;
  lds_byte* lds = (lds_byte*)ring;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  const TilePlace p = place_of<BM, BN>(a, id);
  int32_t left = p.steps;
  const int32_t stages = (left + kStage - 1) / kStage;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = (wave >> 1) * (BM / 2), wj = (wave & 1) * (BN / 2);

  OpA oa;
  OpB ob;
  oa.init(a.A, a.lda, p.i0, a.m - p.i0, p.k0);
  ob.init(a.B, a.ldb, p.j0, a.n - p.j0, p.k0);
  const uint32_t at_a = OpA::fragment_base(wi), at_b = OpB::fragment_base(wj);
  Sums16<FA, FB> sums = {};
  frag fa[2][FA], fb[2][FB];
  // read i of the fragments of a slot's half, into that half's set
  const auto read = [&](lds_byte* slot, int half, int i) {
    if (i < FA) fa[half][i] = OpA::fragment(slot, at_a, i, half);
    else fb[half][i - FA] = OpB::fragment(slot + OpA::kBytes, at_b, i - FA, half);
  };
  const auto product = [&](int half, int c) { mfma_in_place(sums.acc[c / FB][c % FB], fb[half][c % FB], fa[half][c / FB], 0); };

#pragma unroll
  for (int s = 0; s < 2; ++s) {
    oa.load_stage(lds0 + s * kSlot, left);
    ob.load_stage(lds0 + s * kSlot + OpA::kBytes, left);
    left -= kStage;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(waitcnt(OpA::kLoads + OpB::kLoads, 15));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kReads; ++i) read(lds, 0, i);

  for (int32_t t = 0; t < stages; ++t) {
    const uint32_t slot = (uint32_t)(t & 1) * kSlot;
    __builtin_amdgcn_s_waitcnt(waitcnt(63, 0));
    interleave<kReads, kProducts>([&](int i) { read(lds + slot, 1, i); }, [&](int c) { product(0, c); });
    // stage t + 1 has arrived, and every wavefront has all of stage t in registers
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (left < kStage) {
      oa.tail(left);
      ob.tail(left);
    }
    lds_byte* next = lds + (slot ^ kSlot);
    // a read and a load in turn (past the last stage the reads are leftovers that nothing uses)
    constexpr int kOps = kReads > Loads::kOps ? 2 * kReads : 2 * Loads::kOps;
    interleave<kOps, kProducts>(
        [&](int i) {
          if (i % 2 == 0) {
            if (i / 2 < kReads) read(next, 0, i / 2);
          } else if (i / 2 < Loads::kOps) {
            Loads::issue(oa, ob, lds0 + slot, i / 2);
          }
        },
        [&](int c) { product(1, c); });
    oa.advance();
    ob.advance();
    left -= kStage;
  }
  end.template finish<T, BM, BN>(a, ring, sums, p);
}

// The same for smaller tiles and fp32: stages of 64 bytes of a row, a ring of four slots. While the
// products of stage t run, stage t + 1's fragments are read and stages t + 2 .. t + 4 are on their way.
template <typename T, int BM, int BN, bool kAMajor, bool kBMajor, typename End>
__device__ __forceinline__ void ring_tile(const ProductArgs& a, uint32_t id, uint8_t* ring, const End& end) {
  typedef typename Stage<T>::frag frag;
  typedef Operand<T, BM, kAMajor, 1> OpA;
  typedef Operand<T, BN, kBMajor, 1> OpB;
  typedef StageLoads<OpA, OpB> Loads;
  constexpr int kStage = OpA::kSteps, kSlot = OpA::kBytes + OpB::kBytes, kLoads = OpA::kLoads + OpB::kLoads;
  constexpr int FA = BM / 32, FB = BN / 32;  // fragments of a wavefront's BM / 2 x BN / 2
  constexpr int kReads = FA + FB, kProducts = FA * FB * (sizeof(T) == 4 ? 4 : 1);
  lds_byte* lds = (lds_byte*)ring;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  const TilePlace p = place_of<BM, BN>(a, id);
  int32_t left = p.steps;
  const int32_t stages = (left + kStage - 1) / kStage;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = (wave >> 1) * (BM / 2), wj = (wave & 1) * (BN / 2);

  OpA oa;
  OpB ob;
  oa.init(a.A, a.lda, p.i0, a.m - p.i0, p.k0);
  ob.init(a.B, a.ldb, p.j0, a.n - p.j0, p.k0);
  const uint32_t at_a = OpA::fragment_base(wi), at_b = OpB::fragment_base(wj);
  Sums16<FA, FB> sums = {};
  frag fa[2][FA], fb[2][FB];
  const auto read = [&](lds_byte* slot, int to, int i) {
    if (i < FA) fa[to][i] = OpA::fragment(slot, at_a, i);
    else fb[to][i - FA] = OpB::fragment(slot + OpA::kBytes, at_b, i - FA);
  };

#pragma unroll
  for (int s = 0; s < kRing; ++s) {
    oa.load_stage(lds0 + s * kSlot, left);
    ob.load_stage(lds0 + s * kSlot + OpA::kBytes, left);
    left -= kStage;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(waitcnt((kRing - 1) * kLoads, 15));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kReads; ++i) read(lds, 0, i);

  const auto stage = [&](int now, uint32_t slot) {
    // stage t + 1 has arrived (two younger ones may be on their way), and every wavefront has stage t's
    // fragments in registers
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt((kRing - 2) * kLoads, 0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (left < kStage) {
      oa.tail(left);
      ob.tail(left);
    }
    const uint32_t here = lds0 + slot * kSlot;
    lds_byte* next = lds + ((slot + 1) & (kRing - 1)) * kSlot;
    constexpr int kOps = kReads > Loads::kOps ? 2 * kReads : 2 * Loads::kOps;
    interleave<kOps, kProducts>(
        [&](int i) {
          if (i % 2 == 0) {
            if (i / 2 < kReads) read(next, now ^ 1, i / 2);
          } else if (i / 2 < Loads::kOps) {
            Loads::issue(oa, ob, here, i / 2);
          }
        },
        [&](int c) {
          mfma_in_place(sums.acc[c / FB % FA][c % FB], fb[now][c % FB], fa[now][c / FB % FA], c / (FA * FB));
        });
    oa.advance();
    ob.advance();
    left -= kStage;
  };
  // stages in pairs, so that the two sets of fragments keep their registers; where their number is odd
  // the last one's loads all lie beyond the extent and its products add zeros
  for (int32_t t = 0; t < stages; t += 2) {
    stage(0, t & (kRing - 1));
    stage(1, (t + 1) & (kRing - 1));
  }
  end.template finish<T, BM, BN>(a, ring, sums, p);
}

constexpr int ring_bytes(int tile) { return kRing * 2 * tile * 64; }

uint32_t groups_of(const ProductArgs& a) { return (uint32_t)(a.whole + (a.tiles() - a.whole) * a.splits); }

}  // namespace
}  // namespace xtvxy
