// Low-rank adapters of many requests beside the microscaled 4-bit product:
// the part that reads the activations, U[t] = f_i A_i X[t] with i = index[t].
// The product's kernels take it from there (mx4_adapter.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx4_adapter.h"
#include "qamw.h"
#include "qamw_internal.h"

namespace qamw {

// ---------------------------------------------------------------------------
// A workgroup takes 16 tokens, 16 RF ranks and every gridDim.y-th of the
// adapters that these tokens use; its 8 wavefronts split the contraction and
// their sums are added in LDS in a fixed order.  A rows are the product's rows,
// tokens its columns: a token keeps the columns of its own adapter only.
// ---------------------------------------------------------------------------
template <class Ad, int RF>
__global__ __launch_bounds__(kThinThreads) void adapter_shrink_kernel(const typename Ad::E* __restrict__ X, int64_t T, int64_t d,
                                                                      int64_t ldx, const typename Ad::E* __restrict__ A,
                                                                      const float* __restrict__ factors, Adapters ad) {
  typedef typename Ad::E E;
  constexpr int kElems = 16 / sizeof(E), kUnit = 4 * kElems, kBatch = 4;
  __shared__ __align__(16) char red[thin_lds_bytes<RF, 1>()];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * 16 + l16;
  const int r0 = blockIdx.z * 16 * RF;
  int idx[1];
  adapters_of(idx, ad.index, ad.n, t, T);
  const E* x = X + (t < T ? t : 0) * ldx;
  const int64_t units = (d + kUnit - 1) / kUnit, per = (units + kThinWaves - 1) / kThinWaves;
  const int64_t j0 = min(wave * per, units) * kUnit, j1 = min(min(wave * per + per, units) * kUnit, d);
  each_adapter(idx, blockIdx.y, gridDim.y, [&](int use) __attribute__((always_inline)) {
    const bool mine = idx[0] == use;
    const E* a = A + ((int64_t)use * ad.rank + r0 + l16) * d;
    f32x4 acc[RF][1] = {}, ended[RF] = {};
    int steps = 0;
    for (int64_t j = j0; j < j1; j += kBatch * kUnit) {
      i32x4 xf[kBatch], af[kBatch][RF];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t at = j + k * kUnit + kElems * g;
        xf[k] = mine ? load_chunk(x, at, j1) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RF; ++i)
          af[k][i] = r0 + 16 * i + l16 < ad.rank ? load_chunk(a + (int64_t)16 * i * d, at, j1) : i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < RF; ++i) acc[i][0] = Ad::Op::mma(af[k][i], xf[k], acc[i][0], 0, 0, 0);
      if (sizeof(E) == 4 && ++steps % 8 == 0)      // fp32 chains of 512 products (OpF32 says why)
#pragma unroll
        for (int i = 0; i < RF; ++i) ended[i] += acc[i][0], acc[i][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int i = 0; i < RF; ++i) acc[i][0] += ended[i];
    thin_sum(acc, red);
    if (wave || !mine) return;
    const float f = factors ? factors[use] : 1.0f;
#pragma unroll
    for (int i = 0; i < RF; ++i) {
      const int k = r0 + 16 * i + 4 * g;
      if (k >= ad.pitch) continue;                 // whole fours
      f32x4 u = acc[i][0] * f;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = k + e < ad.rank ? u[e] : 0.0f;
      E* to = (E*)const_cast<void*>(ad.U) + t * ad.pitch + k;
      if constexpr (RF == 1) {                     // the other half of a row of 32
        if constexpr (sizeof(E) == 4) *reinterpret_cast<f32x4*>(to + 16) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        else *reinterpret_cast<uint2*>(to + 16) = *reinterpret_cast<uint2*>(to + 16 + T * ad.pitch) = make_uint2(0, 0);
      }
      if constexpr (sizeof(E) == 4) {
        *reinterpret_cast<f32x4*>(to) = u;
      } else {
        const uint32_t h0 = pack_bf16x2(u[0], u[1]), h1 = pack_bf16x2(u[2], u[3]);
        *reinterpret_cast<uint2*>(to) = make_uint2(h0, h1);
        const f32x4 rest = {u[0] - __uint_as_float(h0 << 16), u[1] - __uint_as_float(h0 & 0xffff0000u),
                            u[2] - __uint_as_float(h1 << 16), u[3] - __uint_as_float(h1 & 0xffff0000u)};
        *reinterpret_cast<uint2*>(to + T * ad.pitch) = make_uint2(pack_bf16x2(rest[0], rest[1]), pack_bf16x2(rest[2], rest[3]));
      }
    }
  });
}

// ===========================================================================
// launchers
// ===========================================================================
int64_t adapter_pitch(int64_t rank) { return (rank + 31) / 32 * 32; }
size_t adapter_workspace_bytes(int64_t T, int64_t rank) { return (size_t)T * adapter_pitch(rank) * 4; }
static int64_t rank_tiles(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }
// up to 16 workgroups share the adapters of 16 tokens, where there are few tokens
static int64_t adapter_slots(int64_t T, int64_t n) {
  return std::max<int64_t>(1, std::min<int64_t>({n, 16, tiles_of(4 * kCus, tiles_of(T, 16))}));
}
bool adapter_grid_fits(int64_t T, int64_t rank, int64_t n) {
  return grid_holds(tiles_of(T, 16), kThinThreads) && tiles_of(rank, 16 * rank_tiles(rank)) <= 65535 && n >= 0;
}

template <class Ad, int RF>
static int shrink_as(const void* X, int64_t T, int64_t d, int64_t ldx, const void* A, const float* factors, const Adapters& ad,
                     hipStream_t st) {
  typedef typename Ad::E E;
  const dim3 grid((unsigned)tiles_of(T, 16), (unsigned)adapter_slots(T, ad.n), (unsigned)tiles_of(ad.rank, 16 * RF));
  hipLaunchKernelGGL((adapter_shrink_kernel<Ad, RF>), grid, dim3(kThinThreads), 0, st, (const E*)X, T, d, ldx, (const E*)A,
                     factors, ad);
  return check_launch("adapter_shrink_kernel");
}
template <class Ad>
static int shrink_of(const void* X, int64_t T, int64_t d, int64_t ldx, const void* A, const float* factors, const Adapters& ad,
                     hipStream_t st) {
  const int64_t tiles = rank_tiles(ad.rank);
  if (tiles == 1) return shrink_as<Ad, 1>(X, T, d, ldx, A, factors, ad, st);
  if (tiles == 2) return shrink_as<Ad, 2>(X, T, d, ldx, A, factors, ad, st);
  return shrink_as<Ad, 4>(X, T, d, ldx, A, factors, ad, st);
}
int launch_adapter_shrink(const void* X, int32_t xdt, int64_t T, int64_t d, int64_t ldx, const void* A, const float* factors,
                          const Adapters& ad, hipStream_t st) {
  if (xdt == QAMW_F32) return shrink_of<AdaptersF32>(X, T, d, ldx, A, factors, ad, st);
  return shrink_of<AdaptersBf16>(X, T, d, ldx, A, factors, ad, st);
}

}  // namespace qamw
