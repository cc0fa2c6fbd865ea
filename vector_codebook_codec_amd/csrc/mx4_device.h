// The microscaled 4-bit format on the device (mxfp4.hip states it): element
// types in memory, rows of any length and alignment, a block's scale code and
// codes, and the store of a product's results.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qamw_device.h"
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

// 8 consecutive elements of a row from column j; past the row's end 0 is read
// and nothing written.  Rows start anywhere (an odd row length puts them off
// every boundary): whole groups go as 16-byte accesses of any alignment, which
// the memory pipeline takes, only the last group of a row one by one.
template <class V, class T> __device__ __forceinline__ V load_any(const T* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof v);
  return v;
}
template <class V, class T> __device__ __forceinline__ void store_any(T* p, V v) { __builtin_memcpy(p, &v, sizeof v); }

template <class Mem>
__device__ __forceinline__ void load8(const typename Mem::T* row, int j, int d, float (&x)[8]) {
  if (j + 8 <= d) {
    if constexpr (sizeof(typename Mem::T) == 4) {
      const f32x4 a = load_any<f32x4>(row + j), b = load_any<f32x4>(row + j + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    } else {
      const u32x4 a = load_any<u32x4>(row + j);
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
__device__ __forceinline__ void store8(typename Mem::T* row, int j, int d, const float (&x)[8]) {
  if (j + 8 <= d) {
    if constexpr (sizeof(typename Mem::T) == 4) {
      store_any(row + j, f32x4{x[0], x[1], x[2], x[3]});
      store_any(row + j + 4, f32x4{x[4], x[5], x[6], x[7]});
    } else {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint32_t)Mem::put(x[2 * i]) | ((uint32_t)Mem::put(x[2 * i + 1]) << 16);
      store_any(row + j, v);
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


// results of 4 consecutive channels n of token t
template <class Out>
__device__ __forceinline__ void store_y(typename Out::T* Y, int64_t ldy, int64_t t, int64_t n, int64_t N, f32x4 v) {
  typename Out::T* p = Y + t * ldy + n;
  if (n + 4 <= N) {
    if constexpr (sizeof(typename Out::T) == 4)
      store_any(p, v);
    else
      store_any(p, make_uint2((uint32_t)Out::put(v[0]) | ((uint32_t)Out::put(v[1]) << 16),
                              (uint32_t)Out::put(v[2]) | ((uint32_t)Out::put(v[3]) << 16)));
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) p[r] = Out::put(v[r]);
  }
}

template <class Tl, class Out>
__device__ __forceinline__ void store_tile(typename Out::T* Y, int64_t ldy, int64_t n0, int64_t T, int64_t m0, int64_t N,
                                           f32x4 (&acc)[Tl::TM][Tl::TN], char* lds) {
  typedef typename Out::T E;
  if constexpr (sizeof(E) == 2) {
    tile16_put<Tl>(lds, acc, [](f32x4 v) {
      return make_uint2((uint32_t)Out::put(v[0]) | ((uint32_t)Out::put(v[1]) << 16),
                        (uint32_t)Out::put(v[2]) | ((uint32_t)Out::put(v[3]) << 16));
    });
    tile16_rows<Tl>(lds, [&](int r, int c, u32x4 v) {
      if (n0 + r >= T || m0 + c >= N) return;
      E* p = Y + (n0 + r) * ldy + m0 + c;
      if (m0 + c + 8 <= N) {
        store_any(p, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (m0 + c + e < N) p[e] = (E)(v[e / 2] >> (16 * (e & 1)));
      }
    });
  } else {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
    const int64_t m = m0 + (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4);
    const int64_t t = n0 + (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15);
#pragma unroll
    for (int j = 0; j < Tl::TN; ++j)
      if (t + 16 * j < T)
#pragma unroll
        for (int i = 0; i < Tl::TM; ++i)
          if (m + 16 * i < N) store_y<Out>(Y, ldy, t + 16 * j, m + 16 * i, N, acc[i][j]);
  }
}

}  // namespace qamw
