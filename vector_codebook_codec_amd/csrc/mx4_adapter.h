// Low-rank adapters beside the microscaled 4-bit product: what the product's
// kernels add to their sums before they are rounded and stored,
//     Y[t][n] += sum_k U[t][k] B_i[n][k],   i = index[t],
// with U[t] = f_i A_i X[t] from adapter_shrink_kernel (adapter.hip).  Either
// they multiply U and B themselves or they start from the second term as
// adapter_expand_kernel left it (launch_mx4_matmul says when).
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
  static constexpr bool kOn = false, kDelta = false;
};
struct AdaptersBf16 {
  static constexpr bool kOn = true, kDelta = false;
  typedef uint16_t E;
  typedef OpBf16 Op;
  static constexpr int kStep = 32, kTerms = 2;
};
struct AdaptersF32 {
  static constexpr bool kOn = true, kDelta = false;
  typedef float E;
  typedef OpF32 Op;
  static constexpr int kStep = 16, kTerms = 1;
};
struct AdapterDelta {                              // of either type, multiplied already
  static constexpr bool kOn = false, kDelta = true;
};

// The adapters among the 16 TN tokens whose adapters the lanes hold (lane l:
// token 16 j + l % 16; INT_MAX: none), one after another in the order of their
// first token.
template <int TN>
struct AdapterWalk {
  uint32_t left[TN];                               // tokens of no adapter walked yet
  __device__ __forceinline__ explicit AdapterWalk(const int (&idx)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) left[j] = (uint32_t)__ballot(idx[j] != INT_MAX) & 0xffffu;
  }
  __device__ __forceinline__ int next(const int (&idx)[TN]) {           // INT_MAX: no more
    int use = INT_MAX;
#pragma unroll
    for (int j = TN - 1; j >= 0; --j)
      if (left[j]) use = __builtin_amdgcn_readlane(idx[j], __builtin_ctz(left[j]));
#pragma unroll
    for (int j = 0; j < TN; ++j) left[j] &= ~(uint32_t)__ballot(idx[j] == use);
    return use;
  }
};
template <int TN>
__device__ __forceinline__ void adapters_of(int (&idx)[TN], const int32_t* index, int n, int64_t t, int64_t T) {
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int i = t + 16 * j < T ? index[t + 16 * j] : -1;
    idx[j] = i >= 0 && i < n ? i : INT_MAX;
  }
}

// Chunk k of an adapter's row n of B, n below N or not (then any row), 0 past
// the rank.  Ranks of whole chunks go without a branch around the load: a
// chunk past the rank reads the row's first and is dropped.
template <class E>
__device__ __forceinline__ i32x4 load_rank_chunk(const E* B, int64_t n, int64_t N, int k, int rank) {
  constexpr int kElems = 16 / sizeof(E);
  const E* row = B + (n < N ? n : N - 1) * rank;
  if (rank % kElems) return load_chunk(row, k, rank);
  const i32x4 v = load_any<i32x4>(row + (k < rank ? k : 0));
  return k < rank ? v : i32x4{0, 0, 0, 0};
}
// Columns of a matrix product are independent: a token's sum is simply kept
// where it does not use the adapter at hand, so what that holds (infinities,
// NaN) stays out of it.
template <class Ad>
__device__ __forceinline__ f32x4 add_mine(bool mine, i32x4 b, const i32x4 (&u)[Ad::kTerms], f32x4 acc) {
  f32x4 s = acc;
#pragma unroll
  for (int n = 0; n < Ad::kTerms; ++n) s = Ad::Op::mma(b, u[n], s, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = mine ? s[e] : acc[e];
  return s;
}
template <class Ad>
__device__ __forceinline__ void load_u(i32x4 (&u)[Ad::kTerms], const Adapters& ad, int64_t t, int64_t T, int k) {
  typedef typename Ad::E E;
#pragma unroll
  for (int n = 0; n < Ad::kTerms; ++n) u[n] = *reinterpret_cast<const i32x4*>((const E*)ad.U + (n * T + (t < T ? t : T - 1)) * ad.pitch + k);
}

// acc (fragments of rows m + 16 i by tokens t + 16 j; m and t are this lane's)
// plus the adapters' part; of the adapters the `part`-th of every `parts`.  For
// few fragments: the rows of kBatch adapters are in flight at a time.
template <class Ad, int TM, int TN>
__device__ __forceinline__ void add_adapters(f32x4 (&acc)[TM][TN], const Adapters& ad, int64_t m, int64_t t, int64_t T, int64_t N,
                                             int part, int parts) {
  typedef typename Ad::E E;
  constexpr int kBatch = TM * TN <= 2 ? 8 : 4;
  const int g = (threadIdx.x & (kWave - 1)) >> 4;
  int idx[TN];
  adapters_of(idx, ad.index, ad.n, t, T);
  for (int k0 = 0; k0 < ad.pitch; k0 += Ad::kStep) {
    const int k = k0 + 16 / (int)sizeof(E) * g;    // below the pitch, a multiple of both steps
    AdapterWalk<TN> walk(idx);
    i32x4 u[TN][Ad::kTerms];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int n = 0; n < Ad::kTerms; ++n) {
        const int64_t row = t + 16 * j < T ? t + 16 * j : T - 1;
        u[j][n] = *reinterpret_cast<const i32x4*>((const E*)ad.U + (n * T + row) * ad.pitch + k);
      }
    int place = 0;
    for (bool more = true; more;) {
      int use[kBatch];
      i32x4 b[kBatch][TM];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        do {
          use[x] = walk.next(idx);
        } while (use[x] != INT_MAX && place++ % parts != part);
        more = use[x] != INT_MAX;
        if (more)
#pragma unroll
          for (int i = 0; i < TM; ++i)
            b[x][i] = load_rank_chunk((const E*)ad.B + (int64_t)use[x] * N * ad.rank, m + 16 * i, N, k, ad.rank);
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (use[x] != INT_MAX && __ballot(idx[j] == use[x]))
#pragma unroll
            for (int i = 0; i < TM; ++i) acc[i][j] = add_mine<Ad>(idx[j] == use[x], b[x][i], u[j], acc[i][j]);
    }
  }
}

// The same for the many fragments of a tile, which leave few registers: rows
// m0 + 16 i and tokens t0 + 16 j of the wavefront, bf16 and ranks of whole
// 16-byte chunks.  One adapter after another (mostly there is one); addresses
// are one register each of B and U and scalar offsets, rows past an operand's
// end are other rows or 0 and are not stored.
template <int TM, int TN>
__device__ __forceinline__ void add_adapters_tile(f32x4 (&acc)[TM][TN], const Adapters& ad, int64_t m0, int64_t t0, int64_t T,
                                                  int64_t N) {
  if (m0 >= N || t0 >= T) return;
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  int idx[TN];
  adapters_of(idx, ad.index, ad.n, t0 + l16, T);
  const int rows = (int)(N - m0 < 16 * TM ? N - m0 : 16 * TM), tokens = (int)(T - t0 < 16 * TN ? T - t0 : 16 * TN);
  const uint32_t pu = 2u * ad.pitch, pb = 2u * ad.rank;
  const __amdgpu_buffer_rsrc_t u_hi = buffer_of((const uint16_t*)ad.U + t0 * ad.pitch, tokens * pu),
                               u_lo = buffer_of((const uint16_t*)ad.U + (T + t0) * ad.pitch, tokens * pu);
  AdapterWalk<TN> walk(idx);
  for (int use = walk.next(idx); use != INT_MAX; use = walk.next(idx)) {
    const __amdgpu_buffer_rsrc_t bb = buffer_of((const uint16_t*)ad.B + ((int64_t)use * N + m0) * ad.rank, rows * pb);
    for (int k0 = 0; k0 < ad.rank; k0 += 32) {
      const int k = k0 + 8 * g;
      const uint32_t vb = k < ad.rank ? l16 * pb + 2u * k : kPastEnd, vu = l16 * pu + 2u * k;
      i32x4 b[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) b[i] = load16(bb, vb, 16 * i < rows ? 16u * i * pb : 0u);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const uint32_t at = 16 * j < tokens ? 16u * j * pu : 0u;
        const i32x4 u[2] = {load16(u_hi, vu, at), load16(u_lo, vu, at)};
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[i][j] = add_mine<AdaptersBf16>(idx[j] == use, b[i], u, acc[i][j]);
      }
    }
  }
}

// acc = the second term of Y as it stands in memory: fragments of channels m +
// 16 i (four from there) by tokens t + 16 j, this lane's
template <int TM, int TN>
__device__ __forceinline__ void load_delta(f32x4 (&acc)[TM][TN], const Adapters& ad, int64_t m, int64_t t, int64_t T) {
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if (t + 16 * j < T && m + 16 * i < ad.delta_pitch)
        acc[i][j] = *reinterpret_cast<const f32x4*>(ad.delta + (t + 16 * j) * ad.delta_pitch + m + 16 * i);
}

}  // namespace qamw
