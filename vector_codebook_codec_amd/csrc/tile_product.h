// Matrix products of row-major operands with a shared contraction axis,
//     C[m][n] = sum_k A[m][k] B[n][k],
// as one workgroup's BM x BN tile: the device code that the microscaled 4-bit
// product and the vocabulary cross entropy share.
//
// Operand rows are streams of 16-byte chunks: 8 bf16, 4 fp32 or 32 four-bit
// elements.  A K step is 8 chunks (128 bytes) of every row of both operands,
// copied from global memory straight into LDS (buffer loads with an LDS
// destination).  Chunk c of row r lies at position c ^ ((r >> 1) & 7) of its
// 128-byte LDS row.  The copy writes LDS in lane order, so the permutation is
// applied to the global address.
//
// Matrix-instruction operands: lane l holds row l % 16 of a 16-row fragment
// and, in instruction s (0 or 1) of a K step, chunk 2 q + s with q = 0, 3, 2,
// 1 for l / 16 = 0, 1, 2, 3.  Which k a chunk stands for does not matter as
// long as A and B agree; this order and the permutation above together let
// every group of 16 lanes that a 16-byte LDS read serves at once (rows 0-3
// and 12-15 of one lane group with rows 4-11 of its neighbour, and the other
// way round) fall in 16 different bank groups: with q = l / 16 each read took
// 4 extra cycles.  Results:
// register r of lane l is C[m = 4 (l / 16) + r][n = l % 16] of a 16 x 16 tile,
// so consecutive registers are consecutive rows of A.
//
// Rows past an operand's end and chunks past its row's end read as zero
// (buffer range check): they add nothing whatever the memory behind holds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "qamw_device.h"
#include "qamw_internal.h"

namespace qamw {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStepChunks = 8;                     // 16-byte chunks per operand row and K step
constexpr int kStepBytes = kStepChunks * 16;
constexpr uint32_t kPastEnd = 0x80000000u;         // a byte offset beyond every buffer's range
// (row pitches are at most kMaxRowBytes, so the 256 rows of a tile stay below it)

// One operand of a product; rows start on 16-byte boundaries.
struct Operand {
  const char* p;            // row 0
  int64_t pitch;            // bytes from row to row
  int64_t rows;
  const uint8_t* scale;     // 4-bit operands: one scale code per chunk, rows of scale_pitch bytes
  int64_t scale_pitch;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
// lane l's 16 bytes from offset voff + soff to lds + 16 l
typedef __attribute__((address_space(3))) void* LdsPtr;
__device__ __forceinline__ void copy16_to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)lds, 16, (int)voff, (int)soff, 0, 0);
}

// ---- element types: products of one fragment pair over one chunk per lane
struct OpBf16 {
  static constexpr int kElems = 8;                 // elements per chunk
  static constexpr int kMmas = 1;                  // matrix instructions per chunk
  static constexpr int kChainSteps = 0;            // K steps that one accumulator runs over; 0: all
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ f32x4 mma(i32x4 a, i32x4 b, f32x4 c, int, int, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};
struct OpF32 {
  static constexpr int kElems = 4;
  static constexpr int kMmas = 4;
  // 512 products in a row, then added to a sum of their own: the rounding
  // errors of a chain grow with the square root of its length (bf16's and
  // 4-bit's instructions take 8 and 32 times as many products at once).
  // Logits of rms 2.8 at d = 8192 are off by 1.2e-6; in one chain by 4.6e-6,
  // and their exponentials by as much relative to themselves.  300 x 5003 x
  // 512 takes 24.9 us against 24.8 us, 20 x 3000 x 2048 44.2 us against 43.8 us.
  static constexpr int kChainSteps = 16;
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ f32x4 mma(i32x4 a, i32x4 b, f32x4 c, int, int, int) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
  }
};
struct OpMx4 {
  static constexpr int kElems = 32;
  static constexpr int kMmas = 1;
  static constexpr int kChainSteps = 0;
  static constexpr bool kScaled = true;
  // s selects the byte of the lane's two scale codes
  static __device__ __forceinline__ f32x4 mma(i32x4 a, i32x4 b, f32x4 c, int s, int sa, int sb) {
    const i32x8 x = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, y = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    return s ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 1, sa, 1, sb)
             : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
  }
};

template <class Op, int BM_, int BN_, int WM_, int WN_, int S_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;    // tile, wavefront grid
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;     // 16 x 16 results per wavefront
  static constexpr int kRows = BM + BN;
  static constexpr int kDataBytes = kRows * kStepBytes;
  static constexpr int kScaleBytes = Op::kScaled ? kRows * 16 : 0;         // codes of two K steps
  static_assert(kThreads == (BM == 64 ? 256 : 512), "shape_threads says how many threads a shape has");
  static constexpr int S = S_;                                    // K steps in LDS, a power of two
  static constexpr int kLdsBytes = S * (kDataBytes + kScaleBytes);
  static constexpr int kCopiesA = BM / 8 / kWaves, kCopiesB = BN / 8 / kWaves;   // 8 rows per wavefront copy
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && (8 * kWaves) % 16 == 0, "whole copies");
  static_assert(!Op::kScaled || (BM % kWave == 0 && BN % kWave == 0), "whole scale copies");

  // acc (0 at the call) = the tile (m0, n0) over K steps [step0, step1), step0 even and below
  // step1; kchunks = chunks of a row.  Every thread of the workgroup calls it;
  // lds holds kLdsBytes.
  //
  // S LDS buffers take the K steps in turn.  Fragments are read from LDS
  // half a step before the matrix instructions that use them, so that one
  // barrier a step is enough and stands between two runs of matrix
  // instructions whose operands are already in registers:
  //   read (k, half 1)       | multiply (k, half 0)
  //   wait for the copies of step k + 1, barrier: nobody reads buffer k again
  //   copy step k + S into it; read (k + 1, half 0) | multiply (k, half 1)
  static __device__ __forceinline__ void run(f32x4 (&acc)[TM][TN], const Operand& A, int64_t m0, const Operand& B,
                                             int64_t n0, int kchunks, int step0, int step1, char* lds) {
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t row_bytes = (uint32_t)kchunks * 16u;
    const int64_t ra = A.rows - m0 < BM ? A.rows - m0 : BM, rb = B.rows - n0 < BN ? B.rows - n0 : BN;
    const __amdgpu_buffer_rsrc_t bufa = buffer_of(A.p + m0 * A.pitch, (uint32_t)((ra - 1) * A.pitch) + row_bytes);
    const __amdgpu_buffer_rsrc_t bufb = buffer_of(B.p + n0 * B.pitch, (uint32_t)((rb - 1) * B.pitch) + row_bytes);
    const int crow = 8 * wave + (lane >> 3);                 // this lane's row of the first copy
    const int chunk = (lane & 7) ^ ((crow >> 1) & 7);
    uint32_t va[kCopiesA], vb[kCopiesB];
#pragma unroll
    for (int i = 0; i < kCopiesA; ++i) va[i] = (uint32_t)((crow + 8 * kWaves * i) * A.pitch) + 16u * chunk;
#pragma unroll
    for (int i = 0; i < kCopiesB; ++i) vb[i] = (uint32_t)((crow + 8 * kWaves * i) * B.pitch) + 16u * chunk;

    __amdgpu_buffer_rsrc_t bsa, bsb;
    if constexpr (Op::kScaled) {
      bsa = buffer_of(A.scale + m0 * A.scale_pitch, (uint32_t)(ra * A.scale_pitch));
      bsb = buffer_of(B.scale + n0 * B.scale_pitch, (uint32_t)(rb * B.scale_pitch));
    }
    char* const scales = lds + S * kDataBytes;

    // With S > 2 steps past the last one are copied too, as zeros: the number of copies in flight then is the
    // same in every step.
    auto copy = [&](int step) __attribute__((always_inline)) {
      char* st = lds + ((step - step0) & (S - 1)) * kDataBytes;
      const bool in = (S == 2 || step < step1) && step * kStepChunks + chunk < kchunks;
      const uint32_t soff = S == 2 || step < step1 ? (uint32_t)step * kStepBytes : 0u;   // below every buffer's size
#pragma unroll
      for (int i = 0; i < kCopiesA; ++i)
        copy16_to_lds(bufa, st + (wave + kWaves * i) * 1024, in ? va[i] : kPastEnd, soff);
#pragma unroll
      for (int i = 0; i < kCopiesB; ++i)
        copy16_to_lds(bufb, st + BM * kStepBytes + (wave + kWaves * i) * 1024, in ? vb[i] : kPastEnd, soff);
      if constexpr (Op::kScaled) {
        // 16 codes of a row, those of this step and the next; a scale row is
        // whole 16-byte groups
        if (((step - step0) & 1) == 0 && (S == 2 || step < step1)) {
          char* sc = scales + (((step - step0) >> 1) & (S - 1)) * kScaleBytes;
          const uint32_t ks = (uint32_t)step * kStepChunks;
#pragma unroll
          for (int r0 = 0; r0 < kRows; r0 += kThreads) {
            const int base = r0 + wave * kWave;              // 64 rows, all of one operand
            if (base < BM) copy16_to_lds(bsa, sc + base * 16, (uint32_t)((base + lane) * A.scale_pitch) + ks, 0);
            else if (base < kRows)
              copy16_to_lds(bsb, sc + base * 16, (uint32_t)((base - BM + lane) * B.scale_pitch) + ks, 0);
          }
        }
      }
    };

    const int l16 = lane & 15, pair = -(lane >> 4) & 3;
    // byte offset in a 128-byte row of this lane's chunk of half s; fragments start at multiples of 16 rows
    const int pos[2] = {((2 * pair) ^ ((l16 >> 1) & 7)) * 16, ((2 * pair + 1) ^ ((l16 >> 1) & 7)) * 16};
    const int arow = wm * (BM / WM) + l16, brow = BM + wn * (BN / WN) + l16;
    i32x4 a[2][TM], b[2][TN];
    int sa[TM] = {}, sb[TN] = {}, na[TM] = {}, nb[TN] = {};
    auto fetch = [&](int step, int s) __attribute__((always_inline)) {
      const char* st = lds + ((step - step0) & (S - 1)) * kDataBytes + pos[s];
#pragma unroll
      for (int i = 0; i < TM; ++i) a[s][i] = *reinterpret_cast<const i32x4*>(st + (arow + 16 * i) * kStepBytes);
#pragma unroll
      for (int j = 0; j < TN; ++j) b[s][j] = *reinterpret_cast<const i32x4*>(st + (brow + 16 * j) * kStepBytes);
    };
    auto fetch_scales = [&](int step) __attribute__((always_inline)) {
      if constexpr (Op::kScaled) {
        const int k = step - step0;
        const char* sc = scales + ((k >> 1) & (S - 1)) * kScaleBytes + (k & 1) * 8 + 2 * pair;
#pragma unroll
        for (int i = 0; i < TM; ++i) na[i] = *reinterpret_cast<const uint16_t*>(sc + (arow + 16 * i) * 16);
#pragma unroll
        for (int j = 0; j < TN; ++j) nb[j] = *reinterpret_cast<const uint16_t*>(sc + (brow + 16 * j) * 16);
      }
    };
    auto take_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = na[i];
#pragma unroll
      for (int j = 0; j < TN; ++j) sb[j] = nb[j];
    };
    auto multiply = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = Op::mma(a[s][i], b[s][j], acc[i][j], s, sa[i], sb[j]);
    };
    // One LDS read between every few matrix instructions (bf16 at 8192 x 8192 x
    // 4096: 392 us against 406 us as the compiler orders them).  The scaled
    // instructions run faster as the compiler orders them (T = 11008, 8192 x
    // 4096: 228 us against 235 us).
    auto interleave = [&]() __attribute__((always_inline)) {
      if constexpr (Op::kScaled) return;
      constexpr int kMma = TM * TN * Op::kMmas, kReads = TM + TN;
#pragma unroll
      for (int i = 0; i < kReads; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);               // LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, kMma / kReads, 0);   // matrix instructions
      }
    };

    // sums of the chains that have ended (only where there are several)
    constexpr bool kChains = Op::kChainSteps > 0;
    f32x4 ended[kChains ? TM : 1][kChains ? TN : 1] = {};
#pragma unroll
    for (int k = 0; k < S; ++k)
      if (S > 2 || step0 + k < step1) copy(step0 + k);
    __builtin_amdgcn_s_waitcnt(0x0f70);                      // vmcnt(0): this wavefront's copies are in LDS
    __syncthreads();
    fetch(step0, 0);
    fetch_scales(step0);
    auto one_step = [&](int step) __attribute__((always_inline)) {
      take_scales();
      fetch(step, 1);
      multiply(0);
      interleave();
      // vmcnt: all copies but those of steps k + 2 to k + S - 1 (copies complete in order; those of scale codes
      // come on top, which only makes the wait a little longer)
      constexpr int kLater = (S - 2) * (kCopiesA + kCopiesB);
      static_assert(kLater < 64, "vmcnt has 6 bits");
      __builtin_amdgcn_s_waitcnt(0x0f70 | (kLater & 15) | (kLater >> 4) << 14);
      __syncthreads();
      if (S > 2 || step + S < step1) copy(step + S);
      fetch(step + 1, 0);                                    // past the last step: zero or stale, not used
      fetch_scales(step + 1);
      multiply(1);
      interleave();
    };
    if constexpr (kChains) {
      for (int step = step0; step < step1;) {
        for (const int end = min(step + Op::kChainSteps, step1); step < end; ++step) one_step(step);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) ended[i][j] += acc[i][j], acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = ended[i][j];
    } else {
      for (int step = step0; step < step1; ++step) one_step(step);
    }
    if (S > 2) __builtin_amdgcn_s_waitcnt(0x0f70);           // no copy outlives the call
  }
};

// The tile shapes (qamw_internal.h says when each is taken).  The larger a
// tile, the fewer operand bytes go through LDS per product: at 8192 x 8192 x
// 4096 in bf16, 392 us (1.40 PFLOP/s) and 498 us with 256 and 128 (fp32 uses
// the two smaller ones).  One
// workgroup of 256 x 256, two of 128 x 128 share a CU, of 64 x 64 five with two
// K steps in LDS and two with four.
template <class Op, int kShape> struct ShapeTile;
template <class Op> struct ShapeTile<Op, 0> { typedef Tile<Op, 64, 64, 2, 2, 4> T; };
template <class Op> struct ShapeTile<Op, 1> { typedef Tile<Op, 64, 64, 2, 2> T; };
template <class Op> struct ShapeTile<Op, 2> { typedef Tile<Op, 128, 128, 4, 2> T; };
template <class Op> struct ShapeTile<Op, 3> { typedef Tile<Op, 256, 256, 4, 2> T; };

// f(Tile()) for a shape chosen at run time
template <class Op, class F>
inline int with_shape(int shape, F&& f) {
  if constexpr (!std::is_same<Op, OpF32>::value) {
    if (shape == 3) return f(typename ShapeTile<Op, 3>::T());
    if (shape == 0) return f(typename ShapeTile<Op, 0>::T());
  }
  if (shape == 2) return f(typename ShapeTile<Op, 2>::T());
  return f(typename ShapeTile<Op, 1>::T());
}

// Workgroup -> tile.  Consecutive workgroups go to the 8 XCDs in turn, each
// with an L2 of its own: XCD x takes one contiguous run of the `count` places.
// Places go through groups of 8 tiles of B (n) by all tiles of A (m), n
// fastest, so that the tiles that an XCD works on at one time share rows of
// both operands.
__device__ __forceinline__ int xcd_place(int id, int count) {
  const int x = id % 8, q = count / 8, rem = count % 8;
  return x * q + (x < rem ? x : rem) + id / 8;
}
__device__ __forceinline__ void tile_at(int place, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kGroup = 8;
  const int group = place / (kGroup * tiles_m), in = place % (kGroup * tiles_m);
  const int first = group * kGroup, width = tiles_n - first < kGroup ? tiles_n - first : kGroup;
  tn = first + in % width;
  tm = in / width;
}
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  tile_at(xcd_place(id, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
}

// A tile of 16-bit results [BN rows n][BM columns m] in LDS, to be written out
// in long runs along either axis.  Row n's 16-byte units are permuted by
// f(n), so that all three accesses spread over the banks: 8-byte writes of 16
// consecutive rows, 16-byte reads along a row, and 4-byte reads down 8 rows
// by lanes 8 rows apart.
template <int BM>
struct Tile16 {
  static_assert(BM == 64 || BM >= 128, "f stays below the units of a row");
  static __device__ __forceinline__ int f(int n) {
    if (BM == 64) return (n >> 3) & 7;
    return (n & 1) | ((n >> 3) & 1) << 1 | ((n >> 1 ^ n >> 4) & 1) << 2 | ((n >> 2 ^ n >> 5) & 1) << 3;
  }
  static __device__ __forceinline__ char* at(char* lds, int n, int m) {
    return lds + n * (BM * 2) + (((m >> 3) ^ f(n)) << 4) + (m & 7) * 2;
  }
  // columns m, m + 1 (m even) of rows n .. n + 7 (n a multiple of 8): 8 results of each column
  static __device__ __forceinline__ void columns(char* lds, int n, int m, u32x4& c0, u32x4& c1) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = *reinterpret_cast<const uint32_t*>(at(lds, n + k, m));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c0[k] = __builtin_amdgcn_perm(w[2 * k + 1], w[2 * k], 0x05040100);
      c1[k] = __builtin_amdgcn_perm(w[2 * k + 1], w[2 * k], 0x07060302);
    }
  }
};

// A workgroup's 16-bit tile into LDS (pack: four consecutive results of a row
// to 8 bytes), once nobody reads the operands there any more ...
template <class Tl, class Pack>
__device__ __forceinline__ void tile16_put(char* lds, const f32x4 (&acc)[Tl::TM][Tl::TN], Pack&& pack) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int m = (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4), n = (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < Tl::TN; ++j)
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
      *reinterpret_cast<uint2*>(Tile16<Tl::BM>::at(lds, n + 16 * j, m + 16 * i)) = pack(acc[i][j]);
  __syncthreads();
}
// ... and f(row n, column m, 8 results) over the tile, a run of lanes along a row
template <class Tl, class F>
__device__ __forceinline__ void tile16_rows(char* lds, F&& f) {
  for (int k = threadIdx.x; k < Tl::BN * (Tl::BM / 8); k += Tl::kThreads) {
    const int n = k / (Tl::BM / 8), m = k % (Tl::BM / 8) * 8;
    f(n, m, *reinterpret_cast<const u32x4*>(Tile16<Tl::BM>::at(lds, n, m)));
  }
}

// ---------------------------------------------------------------------------
// Products with few rows of B: bound by reading A once.  A workgroup of 8
// wavefronts takes 16 RF rows of A and all rows of B (at most 16 TF); the
// wavefronts split K and load their fragments straight from global memory in
// matrix-instruction layout, many loads ahead and with no barrier until their
// sums are added, in a fixed order, in LDS.
// ---------------------------------------------------------------------------
constexpr int kThinWaves = 8, kThinThreads = kThinWaves * kWave;
template <int RF, int TF> constexpr int thin_lds_bytes() { return kThinWaves / 2 * RF * TF * kWave * 16; }

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
}

// Sum of the wavefronts' results, in wavefront 0: 4 + 4, 2 + 2, 1 + 1.
template <int RF, int TF>
__device__ __forceinline__ void thin_sum(f32x4 (&acc)[RF][TF], char* lds) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
#pragma unroll
  for (int h = kThinWaves / 2; h; h >>= 1) {
    f32x4* red = reinterpret_cast<f32x4*>(lds) + (wave & (h - 1)) * RF * TF * kWave + lane;
    if (wave >= h && wave < 2 * h)
#pragma unroll
      for (int i = 0; i < RF * TF; ++i) red[i * kWave] = acc[i / TF][i % TF];
    __syncthreads();
    if (wave < h)
#pragma unroll
      for (int i = 0; i < RF * TF; ++i) acc[i / TF][i % TF] += red[i * kWave];
    __syncthreads();
  }
}

// acc of this wavefront's share of K, unscaled operands, 16 rows of each: 4
// chunks of every row a unit, chunk 4 u + l / 16 in lane l; U units a batch,
// the next batch in flight while one is multiplied.
template <class Op, int U>
__device__ __forceinline__ void thin_run(f32x4& acc, const Operand& A, int64_t m0, const Operand& B, int kchunks) {
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t row_bytes = (uint32_t)kchunks * 16u;
  const int64_t ra = A.rows - m0 < 16 ? A.rows - m0 : 16;
  const __amdgpu_buffer_rsrc_t bufa = buffer_of(A.p + m0 * A.pitch, (uint32_t)((ra - 1) * A.pitch) + row_bytes);
  const __amdgpu_buffer_rsrc_t bufb = buffer_of(B.p, (uint32_t)((B.rows - 1) * B.pitch) + row_bytes);
  const uint32_t va = (uint32_t)l16 * (uint32_t)A.pitch + 16u * g, vb = (uint32_t)l16 * (uint32_t)B.pitch + 16u * g;
  const int units = (kchunks + 3) / 4, per = (units + kThinWaves - 1) / kThinWaves;
  const int u0 = min(wave * per, units), u1 = min(u0 + per, units);
  i32x4 a[2][U], b[2][U];
  auto load = [&](int u, auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const bool in = u + k < u1 && 4 * (u + k) + g < kchunks;
      const uint32_t soff = u + k < u1 ? (uint32_t)(u + k) * 64u : 0u;      // below every buffer's size
      a[S][k] = load16(bufa, in ? va : kPastEnd, soff);
      b[S][k] = load16(bufb, in ? vb : kPastEnd, soff);
    }
  };
  auto multiply = [&](auto set) __attribute__((always_inline)) {
    constexpr int S = decltype(set)::value;
#pragma unroll
    for (int k = 0; k < U; ++k) acc = Op::mma(a[S][k], b[S][k], acc, 0, 0, 0);
  };
  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;
  load(u0, S0());
  for (int u = u0; u < u1; u += 2 * U) {
    load(u + U, S1());
    multiply(S0());
    load(u + 2 * U, S0());
    multiply(S1());
  }
}

}  // namespace qamw
