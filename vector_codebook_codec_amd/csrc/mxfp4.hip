// Microscaled 4-bit floating point: quantisation, dequantisation and the
// product of two quantised operands on the scaled matrix instructions.
//
// A row is cut into blocks of 32 consecutive elements.  A block holds one
// power-of-two scale 2^e, stored as the code e + 127, and 32 elements of one
// sign, two exponent and one mantissa bit, with the magnitudes
// {0, 1/2, 1, 3/2, 2, 3, 4, 6}:
//     m = max |v|,   e = max(floor(log2 m) - 2, -127)       (m = 0: e = -127)
//     element = v 2^-e rounded to nearest, ties to even, beyond 6 to 6.
// The largest element of a block is thus in [4, 8) before it is rounded.  A
// block with an infinity or a NaN gets the code 255, and every value of it
// reads back as NaN.  Elements past the end of a row count as 0.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "qamw.h"
#include "qamw_device.h"
#include "qamw_internal.h"
#include "tile_product.h"

namespace qamw {

// ---- element types in memory
struct MemF32 {
  typedef float T;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
struct MemBf16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)f32_to_bf16_bits(v); }
};
struct MemF16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};

// 8 consecutive elements of a row from column j: as 16-byte loads where the
// launcher found every row 16-byte aligned and the columns are all there,
// else one by one, with 0 past the row's end.
template <class Mem>
__device__ __forceinline__ void load8(const typename Mem::T* row, int j, int d, bool wide, float (&x)[8]) {
  if (wide && j + 8 <= d) {
    if constexpr (sizeof(typename Mem::T) == 4) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(row + j), b = *reinterpret_cast<const f32x4*>(row + j + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4*>(row + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = Mem::get((uint16_t)(a[i] & 0xffffu));
        x[2 * i + 1] = Mem::get((uint16_t)(a[i] >> 16));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = j + i < d ? Mem::get(row[j + i]) : 0.0f;
  }
}
template <class Mem>
__device__ __forceinline__ void store8(typename Mem::T* row, int j, int d, bool wide, const float (&x)[8]) {
  if (wide && j + 8 <= d) {
    if constexpr (sizeof(typename Mem::T) == 4) {
      *reinterpret_cast<f32x4*>(row + j) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(row + j + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint32_t)Mem::put(x[2 * i]) | ((uint32_t)Mem::put(x[2 * i + 1]) << 16);
      *reinterpret_cast<u32x4*>(row + j) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < d) row[j + i] = Mem::put(x[i]);
  }
}

// the larger of a value over the four lanes of a quad, in every lane
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true);   // lanes 1 0 3 2
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true);   // lanes 2 3 0 1
  return v > b ? v : b;
}

// Scale code of a block from its largest |v|, as fp32 bits: exponent field - 2,
// not below 0 (subnormal and tiny blocks); 255 for infinities and NaN.
__device__ __forceinline__ uint32_t scale_code(uint32_t max_bits) {
  const uint32_t e = max_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// The conversions read the scale's exponent field alone, so code 0 as the
// fp32 bits 0 stands for 2^-127 there, as it does in the format.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], uint32_t code) {
  if (code == 255u) return 0u;
  const float s = __uint_as_float(code << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
}
__device__ __forceinline__ void decode8(uint32_t c, uint32_t code, float (&x)[8]) {
  const float s = __uint_as_float(code << 23);           // code 255: NaN
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
                e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = e.x, x[5] = e.y, x[6] = f.x, x[7] = f.y;
}

// ---------------------------------------------------------------------------
// Quantisation: a lane holds 8 elements, a quad of lanes a block.  Bound by
// memory: every element is read once and its half byte written once.
// A workgroup is blockDim.x lanes along a row by blockDim.y rows.
// ---------------------------------------------------------------------------
template <class In, class Val>
__global__ __launch_bounds__(kBlockThreads) void mx4_quantize_kernel(
    const typename In::T* __restrict__ W, int64_t N, int d, int64_t ldw, bool wide_in, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales, int nb, int scale_pitch, typename Val::T* __restrict__ values, int64_t ldv,
    bool wide_val) {
  const int per_row = 4 * nb;                                             // lanes of a row
  for (int64_t n = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; n < N; n += (int64_t)gridDim.y * blockDim.y) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;                  // whole quads are in or out
    if (u >= per_row) continue;
    float x[8];
    load8<In>(W + n * ldw, 8 * u, d, wide_in, x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    const uint32_t code = scale_code(quad_max(m));
    const uint32_t c = encode8(x, code);
    *reinterpret_cast<uint32_t*>(codes + n * (int64_t)nb * 16 + 4 * u) = c;
    uint8_t* srow = scales + n * scale_pitch;
    if ((u & 3) == 0) {
      srow[u >> 2] = (uint8_t)code;
      if (u == per_row - 4)
        for (int k = nb; k < scale_pitch; ++k) srow[k] = 0;
    }
    if (values) {
      decode8(c, code, x);
      store8<Val>(values + n * ldv, 8 * u, d, wide_val, x);
    }
  }
}

template <class Out>
__global__ __launch_bounds__(kBlockThreads) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                       const uint8_t* __restrict__ scales, int64_t N,
                                                                       int d, int nb, int scale_pitch,
                                                                       typename Out::T* __restrict__ W, int64_t ldo,
                                                                       bool wide) {
  const int per_row = 4 * nb;
  for (int64_t n = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; n < N; n += (int64_t)gridDim.y * blockDim.y) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= per_row) continue;
    float x[8];
    decode8(*reinterpret_cast<const uint32_t*>(codes + n * (int64_t)nb * 16 + 4 * u), scales[n * scale_pitch + (u >> 2)], x);
    store8<Out>(W + n * ldo, 8 * u, d, wide, x);
  }
}

// ---------------------------------------------------------------------------
// Y[t][n] = sum_k X^[t][k] W^[n][k] on v_mfma_scale_f32_16x16x128: the
// instruction multiplies 128 four-bit products per result and applies both
// blocks' scales, so nothing is decoded.  Weights are the A operand: a lane
// then holds 4 consecutive channels n of one token.
// ---------------------------------------------------------------------------
template <class Out>
__device__ __forceinline__ void store_y(typename Out::T* Y, int64_t ldy, int64_t t, int64_t n, int64_t N, bool wide,
                                        f32x4 v) {
  typename Out::T* p = Y + t * ldy + n;
  if (wide && n + 4 <= N) {
    if constexpr (sizeof(typename Out::T) == 4)
      *reinterpret_cast<f32x4*>(p) = v;
    else
      *reinterpret_cast<uint2*>(p) = make_uint2((uint32_t)Out::put(v[0]) | ((uint32_t)Out::put(v[1]) << 16),
                                                (uint32_t)Out::put(v[2]) | ((uint32_t)Out::put(v[3]) << 16));
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) p[r] = Out::put(v[r]);
  }
}

template <class Tl, class Out>
__global__ __launch_bounds__(Tl::kThreads) void mx4_matmul_kernel(Operand W, Operand X, int kchunks, int tiles_m,
                                                                  int tiles_n, typename Out::T* __restrict__ Y,
                                                                  int64_t ldy, bool wide) {
  extern __shared__ __align__(1024) char tile_lds[];
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * Tl::BM, n0 = (int64_t)tn * Tl::BN;
  f32x4 acc[Tl::TM][Tl::TN] = {};
  Tl::run(acc, W, m0, X, n0, kchunks, 0, (kchunks + kStepChunks - 1) / kStepChunks, tile_lds);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int64_t m = m0 + (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4);
  const int64_t t = n0 + (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15);
#pragma unroll
  for (int j = 0; j < Tl::TN; ++j)
    if (t + 16 * j < X.rows)
#pragma unroll
      for (int i = 0; i < Tl::TM; ++i)
        if (m + 16 * i < W.rows) store_y<Out>(Y, ldy, t + 16 * j, m + 16 * i, W.rows, wide, acc[i][j]);
}

// ===========================================================================
// launchers
// ===========================================================================
static void row_grid(int64_t N, int per_row, dim3* grid, dim3* block) {
  const int bx = std::min(kBlockThreads, (per_row + 63) / 64 * 64), by = kBlockThreads / bx;
  *block = dim3((unsigned)bx, (unsigned)by);
  *grid = dim3((unsigned)((per_row + bx - 1) / bx), (unsigned)std::min<int64_t>((N + by - 1) / by, 65535));
}
static bool wide_rows(const void* p, int64_t ld, int es) { return aligned16(p) && (ld * es) % 16 == 0; }

template <class In, class Val>
static int quantize_as(const void* W, int64_t N, int d, int64_t ldw, uint8_t* codes, uint8_t* scales, void* values,
                       int64_t ldv, hipStream_t st) {
  dim3 grid, block;
  const int nb = (int)mx4_blocks(d);
  row_grid(N, 4 * nb, &grid, &block);
  hipLaunchKernelGGL((mx4_quantize_kernel<In, Val>), grid, block, 0, st, (const typename In::T*)W, N, d, ldw,
                     wide_rows(W, ldw, sizeof(typename In::T)), codes, scales, nb, (int)mx4_scale_bytes(d),
                     (typename Val::T*)values, ldv, wide_rows(values, ldv, sizeof(typename Val::T)));
  return check_launch("mx4_quantize_kernel");
}
template <class In>
static int quantize_from(const void* W, int64_t N, int d, int64_t ldw, uint8_t* codes, uint8_t* scales, void* values,
                         int32_t vdt, int64_t ldv, hipStream_t st) {
  if (vdt == QAMW_F32) return quantize_as<In, MemF32>(W, N, d, ldw, codes, scales, values, ldv, st);
  if (vdt == QAMW_F16) return quantize_as<In, MemF16>(W, N, d, ldw, codes, scales, values, ldv, st);
  return quantize_as<In, MemBf16>(W, N, d, ldw, codes, scales, values, ldv, st);
}
int launch_mx4_quantize(const void* W, int32_t wdt, int64_t N, int d, int64_t ldw, uint8_t* codes, uint8_t* scales,
                        void* values, int32_t vdt, int64_t ldv, hipStream_t st) {
  if (wdt == QAMW_F32) return quantize_from<MemF32>(W, N, d, ldw, codes, scales, values, vdt, ldv, st);
  if (wdt == QAMW_F16) return quantize_from<MemF16>(W, N, d, ldw, codes, scales, values, vdt, ldv, st);
  return quantize_from<MemBf16>(W, N, d, ldw, codes, scales, values, vdt, ldv, st);
}

template <class Out>
static int dequantize_to(const uint8_t* codes, const uint8_t* scales, int64_t N, int d, void* W, int64_t ldo,
                         hipStream_t st) {
  dim3 grid, block;
  const int nb = (int)mx4_blocks(d);
  row_grid(N, 4 * nb, &grid, &block);
  hipLaunchKernelGGL((mx4_dequantize_kernel<Out>), grid, block, 0, st, codes, scales, N, d, nb, (int)mx4_scale_bytes(d),
                     (typename Out::T*)W, ldo, wide_rows(W, ldo, sizeof(typename Out::T)));
  return check_launch("mx4_dequantize_kernel");
}
int launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t N, int d, void* W, int32_t odt,
                          int64_t ldo, hipStream_t st) {
  if (odt == QAMW_F32) return dequantize_to<MemF32>(codes, scales, N, d, W, ldo, st);
  if (odt == QAMW_F16) return dequantize_to<MemF16>(codes, scales, N, d, W, ldo, st);
  return dequantize_to<MemBf16>(codes, scales, N, d, W, ldo, st);
}

template <class Tl, class Out>
static int matmul_tiled(const Operand& W, const Operand& X, int kchunks, void* Y, int64_t ldy, hipStream_t st) {
  const int tiles_m = (int)tiles_of(W.rows, Tl::BM), tiles_n = (int)tiles_of(X.rows, Tl::BN);
  const bool wide = ldy % 4 == 0 && (uintptr_t)Y % (4 * sizeof(typename Out::T)) == 0;
  auto kernel = mx4_matmul_kernel<Tl, Out>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles_m * tiles_n)), dim3(Tl::kThreads), Tl::kLdsBytes, st, W, X, kchunks,
                     tiles_m, tiles_n, (typename Out::T*)Y, ldy, wide);
  return check_launch("mx4_matmul_kernel");
}
template <class Out>
static int matmul_to(const Operand& W, const Operand& X, int kchunks, void* Y, int64_t ldy, hipStream_t st) {
  return large_tiles_pay(W.rows, X.rows) ? matmul_tiled<LargeTile<OpMx4>, Out>(W, X, kchunks, Y, ldy, st)
                                         : matmul_tiled<SmallTile<OpMx4>, Out>(W, X, kchunks, Y, ldy, st);
}
int launch_mx4_matmul(const void* X, int32_t xdt, int64_t T, int d, int64_t ldx, const uint8_t* wcodes,
                      const uint8_t* wscales, int64_t N, void* Y, int32_t ydt, int64_t ldy, void* ws, hipStream_t st) {
  const int nb = (int)mx4_blocks(d);
  uint8_t* xcodes = (uint8_t*)ws;
  uint8_t* xscales = xcodes + round_up((size_t)T * nb * 16, 256);
  const int rc = launch_mx4_quantize(X, xdt, T, d, ldx, xcodes, xscales, nullptr, QAMW_BF16, 0, st);
  if (rc) return rc;
  const Operand w = {(const char*)wcodes, (int64_t)nb * 16, N, wscales, mx4_scale_bytes(d)};
  const Operand x = {(const char*)xcodes, (int64_t)nb * 16, T, xscales, mx4_scale_bytes(d)};
  return ydt == QAMW_F32 ? matmul_to<MemF32>(w, x, nb, Y, ldy, st) : matmul_to<MemBf16>(w, x, nb, Y, ldy, st);
}

}  // namespace qamw
