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
  constexpr int kElems = 16 / sizeof(E), kUnit = 4 * kElems, kBatch = RF == 1 ? 16 : RF == 2 ? 8 : 4;
  __shared__ __align__(16) char red[thin_lds_bytes<RF, 1>()];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * 16 + l16;
  const int r0 = blockIdx.z * 16 * RF;
  int idx[1];
  adapters_of(idx, ad.index, ad.n, t, T);
  // rows past the last token or the rank are read as row 0: their results are dropped
  const E* x = X + (t < T ? t : 0) * ldx;
  // a lane's chunks are neighbours in pairs, so that the lines of 128 bytes are read at once
  auto chunk = [&](int k) { return (k / 2 * 8 + 2 * g + k % 2) * kElems; };
  const int64_t units = (d + 2 * kUnit - 1) / (2 * kUnit), per = (units + kThinWaves - 1) / kThinWaves;
  const int64_t j0 = min(wave * per, units) * 2 * kUnit, j1 = min(min(wave * per + per, units) * 2 * kUnit, d);
  AdapterWalk<1> walk(idx);
  for (int place = 0;; ++place) {
    const int use = walk.next(idx);
    if (use == INT_MAX) return;
    if (place % gridDim.y != blockIdx.y) continue;
    const bool mine = idx[0] == use;
    const E* a[RF];
#pragma unroll
    for (int i = 0; i < RF; ++i) a[i] = A + ((int64_t)use * ad.rank + (r0 + 16 * i + l16 < ad.rank ? r0 + 16 * i + l16 : 0)) * d;
    f32x4 acc[RF][1] = {}, ended[RF] = {};
    auto multiply = [&](const i32x4 (&xf)[kBatch], const i32x4 (&af)[kBatch][RF]) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < RF; ++i) acc[i][0] = Ad::Op::mma(af[k][i], xf[k], acc[i][0], 0, 0, 0);
    };
    int steps = 0;
    int64_t j = j0;
    i32x4 xf[kBatch], af[kBatch][RF];
    for (; j + kBatch * kUnit <= j1; j += kBatch * kUnit) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        xf[k] = load_any<i32x4>(x + j + chunk(k));
#pragma unroll
        for (int i = 0; i < RF; ++i) af[k][i] = load_any<i32x4>(a[i] + j + chunk(k));
      }
      multiply(xf, af);
      if (sizeof(E) == 4 && ++steps % (512 / (kBatch * kUnit)) == 0)      // fp32 chains of 512 products (OpF32 says why)
#pragma unroll
        for (int i = 0; i < RF; ++i) ended[i] += acc[i][0], acc[i][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (j < j1) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        xf[k] = load_chunk(x, j + chunk(k), j1);
#pragma unroll
        for (int i = 0; i < RF; ++i) af[k][i] = load_chunk(a[i], j + chunk(k), j1);
      }
      multiply(xf, af);
    }
#pragma unroll
    for (int i = 0; i < RF; ++i) acc[i][0] += ended[i];
    thin_sum(acc, red);
    if (wave || !mine) continue;
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
  }
}

// ---------------------------------------------------------------------------
// The adapters' part of Y in fp32: a wavefront takes 16 tokens by 32 channels.
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 256, kExpandRows = 32 * kExpandThreads / kWave;
template <class Ad>
__global__ __launch_bounds__(kExpandThreads) void adapter_expand_kernel(Adapters ad, int64_t T, int64_t N, float* __restrict__ delta) {
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * kExpandRows + (threadIdx.x >> 6) * 32;
  if (m0 >= N) return;
  for (int64_t t = (int64_t)blockIdx.y * 16 + l16; t - l16 < T; t += (int64_t)gridDim.y * 16) {
    f32x4 acc[2][1] = {};
    add_adapters<Ad>(acc, ad, m0 + l16, t, T, N, 0, 1);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (t < T && m0 + 16 * i + 4 * g < ad.delta_pitch)
        *reinterpret_cast<f32x4*>(delta + t * ad.delta_pitch + m0 + 16 * i + 4 * g) = acc[i][0];
  }
}

// ===========================================================================
// launchers
// ===========================================================================
int64_t adapter_pitch(int64_t rank) { return (rank + 31) / 32 * 32; }
// U, and the adapters' part of Y where that is written
size_t adapter_workspace_bytes(int64_t T, int64_t N, int32_t dt, int64_t rank) {
  return adapter_u_bytes(T, rank) + (adapters_in_delta(T, N, dt, rank) ? (size_t)T * adapter_delta_pitch(N) * sizeof(float) : 0);
}
static int64_t rank_tiles(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }
// workgroups that share the adapters of 16 tokens, up to 16 where there are few tokens
static int64_t adapter_slots(int64_t T, int64_t n) {
  return std::max<int64_t>(1, std::min<int64_t>({n, 16, tiles_of(2 * kCus, tiles_of(T, 16))}));
}
bool adapter_grid_fits(int64_t T, int64_t N, int64_t rank) {
  return grid_holds(tiles_of(T, 16), kThinThreads) && tiles_of(rank, 16 * rank_tiles(rank)) <= 65535 &&
         grid_holds(tiles_of(N, kExpandRows), kExpandThreads) && tiles_of(T, 16) <= (int64_t(1) << 27);
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

int launch_adapter_expand(int32_t dt, int64_t T, int64_t N, const Adapters& ad, hipStream_t st) {
  const dim3 grid((unsigned)tiles_of(N, kExpandRows), (unsigned)std::min<int64_t>(tiles_of(T, 16), 65535));
  auto kernel = dt == QAMW_F32 ? adapter_expand_kernel<AdaptersF32> : adapter_expand_kernel<AdaptersBf16>;
  hipLaunchKernelGGL(kernel, grid, dim3(kExpandThreads), 0, st, ad, T, N, const_cast<float*>(ad.delta));
  return check_launch("adapter_expand_kernel");
}

}  // namespace qamw
