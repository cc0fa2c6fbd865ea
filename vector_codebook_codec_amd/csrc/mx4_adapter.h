// Low-rank adapters beside the microscaled 4-bit product: what the product's
// kernels add to their sums before they are rounded and stored,
//     Y[t][n] += sum_k U[t][k] B_i[n][k],   i = index[t],
// with U[t] = f_i A_i X[t] from the kernels of adapter.hip.  Either
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

// The adapters' types.  U in bf16 goes as two numbers (2^-16 of it) where the
// result is bf16 and as three (2^-24) where it is fp32; a step is what one load
// of 16 bytes a lane covers.
struct NoAdapters {
  static constexpr bool kOn = false, kDelta = false;
};
struct AdaptersBf16 {
  static constexpr bool kOn = true, kDelta = false;
  typedef uint16_t E;
  typedef OpBf16 Op;
  static constexpr int kStep = 32, kTerms = 2;
};
struct AdaptersBf16x3 : AdaptersBf16 {
  static constexpr int kTerms = 3;
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

// The adapters among the tokens whose adapters the lanes hold (INT_MAX: none),
// `n` registers of one token a lane in the first kLanes lanes, one after
// another in the order of their first token.
template <int n, int kLanes>
struct AdapterWalk {
  uint64_t left[n];                                // tokens of no adapter walked yet
  __device__ __forceinline__ explicit AdapterWalk(const int (&idx)[n]) {
#pragma unroll
    for (int j = 0; j < n; ++j) left[j] = __ballot(idx[j] != INT_MAX) & (~0ull >> (64 - kLanes));
  }
  __device__ __forceinline__ int next(const int (&idx)[n]) {            // INT_MAX: no more
    int use = INT_MAX;
#pragma unroll
    for (int j = n - 1; j >= 0; --j)
      if (left[j]) use = __builtin_amdgcn_readlane(idx[j], __builtin_ctzll(left[j]));
#pragma unroll
    for (int j = 0; j < n; ++j) left[j] &= ~__ballot(idx[j] == use);
    return use;
  }
};
// lane l: the adapters of tokens t + 16 j, t its own
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
// a lane's chunk of U: its parts, read at once (those that are not there are
// the last one again), then added in a fixed order
template <class Ad>
struct ChunkOfU {
  static constexpr int kQuads = sizeof(typename Ad::E) == 4 ? 1 : 2;
  f32x4 part[kMostAdapterParts][kQuads];
  __device__ __forceinline__ void load(const Adapters& ad, int64_t t, int64_t T, int k) {
#pragma unroll
    for (int p = 0; p < kMostAdapterParts; ++p)
#pragma unroll
      for (int n = 0; n < kQuads; ++n)
        part[p][n] = *reinterpret_cast<const f32x4*>(ad.u_parts + ((p < ad.parts ? p : ad.parts - 1) * T + t) * ad.pitch + k + 4 * n);
  }
  __device__ __forceinline__ void add(i32x4 (&u)[Ad::kTerms], int parts, float factor) const {
    f32x4 s[kQuads];
#pragma unroll
    for (int n = 0; n < kQuads; ++n) s[n] = part[0][n];
#pragma unroll
    for (int p = 1; p < kMostAdapterParts; ++p)
      if (p < parts)
#pragma unroll
        for (int n = 0; n < kQuads; ++n) s[n] += part[p][n];
#pragma unroll
    for (int n = 0; n < kQuads; ++n) s[n] *= factor;
    if constexpr (kQuads == 1) {
      u[0] = __builtin_bit_cast(i32x4, s[0]);
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float x0 = s[n / 2][2 * (n & 1)], x1 = s[n / 2][2 * (n & 1) + 1];
#pragma unroll
        for (int i = 0; i < Ad::kTerms; ++i) {
          const uint32_t h = pack_bf16x2(x0, x1);
          u[i][n] = (int)h;
          x0 -= __uint_as_float(h << 16), x1 -= __uint_as_float(h & 0xffff0000u);
        }
      }
    }
  }
};

// The adapters and factors of a lane's tokens t + 16 j: read ahead of what
// needs them.
template <int TN>
struct TokenAdapters {
  int idx[TN];
  float factor[TN];
  __device__ __forceinline__ TokenAdapters(const Adapters& ad, int64_t t, int64_t T) {
    adapters_of(idx, ad.index, ad.n, t, T);
#pragma unroll
    for (int j = 0; j < TN; ++j) factor[j] = ad.factors && idx[j] != INT_MAX ? ad.factors[idx[j]] : 1.0f;
  }
};
// acc (fragments of rows m + 16 i by tokens t + 16 j; m and t are this lane's)
// plus the adapters' part; of the adapters the `part`-th of every `parts`.  For
// few fragments: the rows of kBatch adapters are in flight at a time.  Returns
// whether the lane's (last) token had one of these adapters.
template <class Ad, int kBatch, int TM, int TN>
__device__ __forceinline__ bool add_adapters(f32x4 (&acc)[TM][TN], const Adapters& ad, const TokenAdapters<TN>& own, int64_t m,
                                             int64_t t, int64_t T, int64_t N, int part, int parts) {
  typedef typename Ad::E E;
  const int g = (threadIdx.x & (kWave - 1)) >> 4;
  bool had = false;
  for (int k0 = 0; k0 < ad.pitch; k0 += Ad::kStep) {
    const int k = k0 + 16 / (int)sizeof(E) * g;    // below the pitch, a multiple of both steps
    ChunkOfU<Ad> chunk[TN];
    i32x4 u[TN][Ad::kTerms];
#pragma unroll
    for (int j = 0; j < TN; ++j) chunk[j].load(ad, t + 16 * j < T ? t + 16 * j : T - 1, T, k);
    AdapterWalk<TN, 16> walk(own.idx);
    int place = part;
    bool ready = false;
    for (bool more = true; more;) {
      int use[kBatch];
      i32x4 b[kBatch][TM];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        for (;; --place) {
          use[x] = walk.next(own.idx);
          if (use[x] == INT_MAX || !place) break;
        }
        place = parts - 1;
        more = use[x] != INT_MAX;
        if (more)
#pragma unroll
          for (int i = 0; i < TM; ++i)
            b[x][i] = load_rank_chunk((const E*)ad.B + (int64_t)use[x] * N * ad.rank, m + 16 * i, N, k, ad.rank);
      }
      if (!ready) {                                // U's parts and the first rows of B are under way together
        ready = true;
#pragma unroll
        for (int j = 0; j < TN; ++j) chunk[j].add(u[j], ad.parts, own.factor[j]);
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (use[x] != INT_MAX && __ballot(own.idx[j] == use[x])) {
            had |= own.idx[j] == use[x];
#pragma unroll
            for (int i = 0; i < TM; ++i) acc[i][j] = add_mine<Ad>(own.idx[j] == use[x], b[x][i], u[j], acc[i][j]);
          }
    }
  }
  return had;
}

// The same for a whole tile, bf16 and ranks of whole 16-byte chunks: 64 ranks
// of U for all its tokens and of B for all its channels are copied to LDS (in
// the order of tile_product.h's operands), one adapter after another; mostly
// there is one.  Every thread of the workgroup calls it; lds holds kLdsBytes of the tile.
template <class Ad, class Tl>
__device__ __forceinline__ void add_adapters_tile(f32x4 (&acc)[Tl::TM][Tl::TN], const Adapters& ad, int64_t m0, int64_t t0, int64_t T,
                                                  int64_t N, char* lds) {
  static_assert((Ad::kTerms * Tl::BN + Tl::BM) * kStepBytes <= Tl::kLdsBytes, "U and B of 64 ranks");
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / Tl::WN, wn = wave % Tl::WN;
  const int rows = (int)(N - m0 < Tl::BM ? N - m0 : Tl::BM), tokens = (int)(T - t0 < Tl::BN ? T - t0 : Tl::BN);
  const uint32_t pu = 2u * ad.pitch, pb = 2u * ad.rank;
  // all tokens of the tile, to walk over; this lane's own, to keep sums by
  int all[Tl::BN / kWave], idx[Tl::TN];
#pragma unroll
  for (int j = 0; j < Tl::BN / kWave; ++j) {
    const int t = lane + kWave * j, i = t < tokens ? ad.index[t0 + t] : -1;
    all[j] = i >= 0 && i < ad.n ? i : INT_MAX;
  }
  adapters_of(idx, ad.index, ad.n, t0 + wn * (Tl::BN / Tl::WN) + l16, T);
  const int crow = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ ((crow >> 1) & 7);
  char *const lds_u = lds, *const lds_b = lds + Ad::kTerms * Tl::BN * kStepBytes;
  for (int k0 = 0; k0 < ad.rank; k0 += 64) {
    const int k = k0 + 8 * chunk;
    __syncthreads();                               // nobody reads what LDS held
#pragma unroll
    for (int i = 0; i < Tl::kCopiesB; ++i) {
      const uint32_t at = k < ad.pitch ? (uint32_t)(crow + 8 * Tl::kWaves * i) * pu + 2u * k : kPastEnd;
#pragma unroll
      for (int n = 0; n < Ad::kTerms; ++n)
        copy16_to_lds(buffer_of(ad.u16 + (n * T + t0) * ad.pitch, tokens * pu),
                      lds_u + n * Tl::BN * kStepBytes + (wave + Tl::kWaves * i) * 1024, at, 0);
    }
    AdapterWalk<Tl::BN / kWave, kWave> walk(all);
    bool first = true;
    for (int use = walk.next(all); use != INT_MAX; use = walk.next(all), first = false) {
      if (!first) __syncthreads();                 // nobody reads the last adapter's rows
      const __amdgpu_buffer_rsrc_t bb = buffer_of((const uint16_t*)ad.B + ((int64_t)use * N + m0) * ad.rank, rows * pb);
#pragma unroll
      for (int i = 0; i < Tl::kCopiesA; ++i)
        copy16_to_lds(bb, lds_b + (wave + Tl::kWaves * i) * 1024,
                      k < ad.rank ? (uint32_t)(crow + 8 * Tl::kWaves * i) * pb + 2u * k : kPastEnd, 0);
      __builtin_amdgcn_s_waitcnt(0x0f70);          // vmcnt(0): this wavefront's copies are in LDS
      __syncthreads();
      bool any = false;
#pragma unroll
      for (int j = 0; j < Tl::TN; ++j) any |= idx[j] == use;
      if (!__ballot(any)) continue;
      for (int s = 0; s < 2 && k0 + 32 * s < ad.rank; ++s) {
        // chunk 4 s + g of a row; fragments start at multiples of 16 rows
        const int pos = ((4 * s + g) ^ ((l16 >> 1) & 7)) * 16;
        i32x4 b[Tl::TM];
#pragma unroll
        for (int i = 0; i < Tl::TM; ++i)
          b[i] = *reinterpret_cast<const i32x4*>(lds_b + (wm * (Tl::BM / Tl::WM) + 16 * i + l16) * kStepBytes + pos);
#pragma unroll
        for (int j = 0; j < Tl::TN; ++j) {
          const char* at = lds_u + (wn * (Tl::BN / Tl::WN) + 16 * j + l16) * kStepBytes + pos;
          i32x4 u[Ad::kTerms];
#pragma unroll
          for (int n = 0; n < Ad::kTerms; ++n) u[n] = *reinterpret_cast<const i32x4*>(at + n * Tl::BN * kStepBytes);
#pragma unroll
          for (int i = 0; i < Tl::TM; ++i) acc[i][j] = add_mine<Ad>(idx[j] == use, b[i], u, acc[i][j]);
        }
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
