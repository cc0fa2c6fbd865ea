// Low-rank adapters beside the microscaled 4-bit product: what the product's
// kernels add to their sums before they are rounded and stored,
//     Y[t][n] += sum_k U[t][k] B_i[n][k],   i = index[t],
// with U[t] = f_i A_i X[t] from adapter_shrink_kernel (adapter.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "mx4_device.h"
#include "qamw_device.h"
#include "qamw_internal.h"
#include "tile_product.h"

namespace qamw {

// 16 bytes of a row from column j, 0 past the row's end; rows start anywhere
template <class E>
__device__ __forceinline__ i32x4 load_chunk(const E* row, int64_t j, int64_t d) {
  constexpr int kElems = 16 / sizeof(E);
  if (j + kElems <= d) return load_any<i32x4>(row + j);
  E e[kElems];
#pragma unroll
  for (int i = 0; i < kElems; ++i) e[i] = j + i < d ? row[j + i] : E(0);
  return __builtin_bit_cast(i32x4, e);
}

// The adapters' types.  U in bf16 goes as two numbers, so that only the
// adapters' own rounding is in the result; a step is what one load of 16 bytes
// a lane covers.
struct NoAdapters {
  static constexpr bool kOn = false;
};
struct AdaptersBf16 {
  static constexpr bool kOn = true;
  typedef uint16_t E;
  typedef OpBf16 Op;
  static constexpr int kStep = 32, kTerms = 2;
};
struct AdaptersF32 {
  static constexpr bool kOn = true;
  typedef float E;
  typedef OpF32 Op;
  static constexpr int kStep = 16, kTerms = 1;
};

// Calls f(i) for every adapter among the 16 TN tokens whose adapters the lanes
// hold (lane l: token 16 j + l % 16; INT_MAX: none), in increasing order; of
// these the `part`-th of every `parts`.
template <int TN, class F>
__device__ __forceinline__ void each_adapter(const int (&idx)[TN], int part, int parts, F&& f) {
  int last = -1, place = 0;
  for (;;) {
    int next = INT_MAX;
#pragma unroll
    for (int j = 0; j < TN; ++j) next = idx[j] > last && idx[j] < next ? idx[j] : next;
#pragma unroll
    for (int x = 1; x < 16; x *= 2) next = min(next, __shfl_xor(next, x));
    next = __builtin_amdgcn_readfirstlane(next);
    if (next == INT_MAX) return;
    last = next;
    if (place == part) f(next);
    place = place + 1 == parts ? 0 : place + 1;
  }
}
template <int TN>
__device__ __forceinline__ void adapters_of(int (&idx)[TN], const int32_t* index, int n, int64_t t, int64_t T) {
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int i = t + 16 * j < T ? index[t + 16 * j] : -1;
    idx[j] = i >= 0 && i < n ? i : INT_MAX;
  }
}

// acc (fragments of rows m + 16 i by tokens t + 16 j; m and t are this lane's)
// plus the adapters' part.  Columns of a matrix product are independent, so a
// token's sum is simply kept where it does not use the adapter at hand: what
// that holds (infinities, NaN) stays out of it.
template <class Ad, int TM, int TN>
__device__ __forceinline__ void add_adapters(f32x4 (&acc)[TM][TN], const Adapters& ad, int64_t m, int64_t t, int64_t T, int64_t N,
                                             int part, int parts) {
  typedef typename Ad::E E;
  const int g = (threadIdx.x & (kWave - 1)) >> 4;
  constexpr int kElems = 16 / sizeof(E);
  int idx[TN];
  adapters_of(idx, ad.index, ad.n, t, T);
  each_adapter(idx, part, parts, [&](int use) __attribute__((always_inline)) {
    const E* B = (const E*)ad.B + (int64_t)use * N * ad.rank;
    for (int k = kElems * g; k < ad.pitch; k += Ad::kStep) {             // pitch: a multiple of both steps
      i32x4 b[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        b[i] = m + 16 * i < N ? load_chunk(B + (m + 16 * i) * ad.rank, k, ad.rank) : i32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const bool mine = idx[j] == use;
        if (!__ballot(mine)) continue;
        i32x4 u[Ad::kTerms];
#pragma unroll
        for (int n = 0; n < Ad::kTerms; ++n)
          u[n] = mine ? *reinterpret_cast<const i32x4*>((const E*)ad.U + (n * T + t + 16 * j) * ad.pitch + k) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          f32x4 s = acc[i][j];
#pragma unroll
          for (int n = 0; n < Ad::kTerms; ++n) s = Ad::Op::mma(b[i], u[n], s, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = mine ? s[e] : acc[i][j][e];
        }
      }
    }
  });
}

}  // namespace qamw
