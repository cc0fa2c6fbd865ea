// Matrix products of row-major operands with a shared contraction axis,
//     C[m][n] = sum_k A[m][k] B[n][k],
// as one workgroup's BM x BN tile: the device code that the microscaled 4-bit
// product and the vocabulary cross entropy share.
//
// Operand rows are streams of 16-byte chunks: 8 bf16, 4 fp32 or 32 four-bit
// elements.  A K step is 8 chunks (128 bytes) of every row of both operands,
// copied from global memory straight into LDS (buffer loads with an LDS
// destination).  Chunk c of row r lies at position c ^ ((r >> 1) & 7) of its
// 128-byte LDS row: the 16 rows that a matrix instruction reads at one chunk
// index then fall in 16 different 16-byte bank groups.  The copy writes LDS
// in lane order, so the permutation is applied to the global address.
//
// Matrix-instruction operands: lane l holds row l % 16 of a 16-row fragment
// and, in instruction s (0 or 1) of a K step, chunk 2 (l / 16) + s.  Which k
// a chunk stands for does not matter as long as A and B agree.  Results:
// register r of lane l is C[m = 4 (l / 16) + r][n = l % 16] of a 16 x 16 tile,
// so consecutive registers are consecutive rows of A.
//
// Rows past an operand's end and chunks past its row's end read as zero
// (buffer range check): they add nothing whatever the memory behind holds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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
// lane l's 16 (4) bytes from offset voff + soff to lds + 16 l (4 l)
typedef __attribute__((address_space(3))) void* LdsPtr;
__device__ __forceinline__ void copy16_to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)lds, 16, (int)voff, (int)soff, 0, 0);
}
__device__ __forceinline__ void copy4_to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)lds, 4, (int)voff, (int)soff, 0, 0);
}

// ---- element types: products of one fragment pair over one chunk per lane
struct OpBf16 {
  static constexpr int kElems = 8;                 // elements per chunk
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ f32x4 mma(i32x4 a, i32x4 b, f32x4 c, int, int, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};
struct OpF32 {
  static constexpr int kElems = 4;
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
  static constexpr bool kScaled = true;
  // s selects the byte of the lane's two scale codes
  static __device__ __forceinline__ f32x4 mma(i32x4 a, i32x4 b, f32x4 c, int s, int sa, int sb) {
    const i32x8 x = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, y = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    return s ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 1, sa, 1, sb)
             : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
  }
};

template <class Op, int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;    // tile, wavefront grid
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;     // 16 x 16 results per wavefront
  static constexpr int kRows = BM + BN;
  static constexpr int kDataBytes = kRows * kStepBytes;
  static constexpr int kStageBytes = kDataBytes + (Op::kScaled ? kRows * kStepChunks : 0);
  static constexpr int kLdsBytes = 2 * kStageBytes;
  static constexpr int kCopiesA = BM / 8 / kWaves, kCopiesB = BN / 8 / kWaves;   // 8 rows per wavefront copy
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && (8 * kWaves) % 16 == 0, "whole copies");

  // acc += the tile (m0, n0) over K steps [step0, step1); kchunks = chunks of
  // a row.  Every thread of the workgroup calls it; lds holds kLdsBytes.
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
    constexpr int kSaCopies = Op::kScaled ? (BM * 2 + kThreads - 1) / kThreads : 0;
    constexpr int kSbCopies = Op::kScaled ? (BN * 2 + kThreads - 1) / kThreads : 0;
    if constexpr (Op::kScaled) {
      bsa = buffer_of(A.scale + m0 * A.scale_pitch, (uint32_t)(ra * A.scale_pitch));
      bsb = buffer_of(B.scale + n0 * B.scale_pitch, (uint32_t)(rb * B.scale_pitch));
    }

    auto copy = [&](int step, char* st) __attribute__((always_inline)) {
      const bool in = step * kStepChunks + chunk < kchunks;
      const uint32_t soff = (uint32_t)step * kStepBytes;
#pragma unroll
      for (int i = 0; i < kCopiesA; ++i)
        copy16_to_lds(bufa, st + (wave + kWaves * i) * 1024, in ? va[i] : kPastEnd, soff);
#pragma unroll
      for (int i = 0; i < kCopiesB; ++i)
        copy16_to_lds(bufb, st + BM * kStepBytes + (wave + kWaves * i) * 1024, in ? vb[i] : kPastEnd, soff);
      if constexpr (Op::kScaled) {
        // two dwords (8 codes) per row; a scale row is whole 16-byte groups
        char* sc = st + kDataBytes;
        const uint32_t ks = (uint32_t)step * kStepChunks + 4u * (threadIdx.x & 1);
#pragma unroll
        for (int i = 0; i < kSaCopies; ++i) {
          const int base = i * kThreads + wave * kWave;
          if (base < BM * 2)
            copy4_to_lds(bsa, sc + base * 4, (uint32_t)(((base + lane) >> 1) * A.scale_pitch) + ks, 0);
        }
#pragma unroll
        for (int i = 0; i < kSbCopies; ++i) {
          const int base = i * kThreads + wave * kWave;
          if (base < BN * 2)
            copy4_to_lds(bsb, sc + BM * 8 + base * 4, (uint32_t)(((base + lane) >> 1) * B.scale_pitch) + ks, 0);
        }
      }
    };

    const int l16 = lane & 15, g = lane >> 4;
    // byte offset in a 128-byte row of this lane's chunk of instruction s; fragments start at multiples of 16 rows
    const int pos[2] = {((2 * g) ^ ((l16 >> 1) & 7)) * 16, ((2 * g + 1) ^ ((l16 >> 1) & 7)) * 16};
    const int arow = wm * (BM / WM) + l16, brow = wn * (BN / WN) + l16;

    copy(step0, lds);
    for (int step = step0; step < step1; ++step) {
      char* st = lds + ((step - step0) & 1) * kStageBytes;
      __builtin_amdgcn_s_waitcnt(0x0f70);                    // vmcnt(0): this wavefront's part of the step is in LDS
      __syncthreads();
      if (step + 1 < step1) copy(step + 1, lds + ((step + 1 - step0) & 1) * kStageBytes);
      int sa[TM], sb[TN];
      if constexpr (Op::kScaled) {
        const char* sc = st + kDataBytes;
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = *reinterpret_cast<const uint16_t*>(sc + (arow + 16 * i) * 8 + 2 * g);
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = *reinterpret_cast<const uint16_t*>(sc + (BM + brow + 16 * j) * 8 + 2 * g);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        i32x4 a[TM], b[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
          a[i] = *reinterpret_cast<const i32x4*>(st + (arow + 16 * i) * kStepBytes + pos[s]);
#pragma unroll
        for (int j = 0; j < TN; ++j)
          b[j] = *reinterpret_cast<const i32x4*>(st + (BM + brow + 16 * j) * kStepBytes + pos[s]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = Op::mma(a[i], b[j], acc[i][j], s, Op::kScaled ? sa[i] : 0, Op::kScaled ? sb[j] : 0);
      }
    }
  }
};

// Workgroup -> tile.  Consecutive workgroups go to the 8 XCDs in turn, each
// with an L2 of its own: XCD x takes one contiguous run of tiles, and runs go
// through groups of 8 tiles of B (n) by all tiles of A (m), m fastest inside
// a column of the group, so that the tiles that an XCD works on at one time
// share rows of both operands.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n;
  const int x = id % 8, q = total / 8, rem = total % 8;
  const int t = x * q + (x < rem ? x : rem) + id / 8;
  constexpr int kGroup = 8;
  const int group = t / (kGroup * tiles_m), in = t % (kGroup * tiles_m);
  const int first = group * kGroup, width = tiles_n - first < kGroup ? tiles_n - first : kGroup;
  tn = first + in % width;
  tm = in / width;
}

}  // namespace qamw
