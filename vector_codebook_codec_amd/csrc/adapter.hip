// Low-rank adapters of many requests beside the microscaled 4-bit product:
// the part that reads the activations, U[t] = f_i A_i X[t] with i = index[t],
// and U B_i^T as a matrix where the product takes it so (mx4_adapter.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx4_adapter.h"
#include "qamw.h"
#include "qamw_internal.h"

namespace qamw {

// ---------------------------------------------------------------------------
// Few tokens, and operands of any alignment.  A workgroup takes 16 tokens, 16
// RF ranks, one of `parts` shares of the contraction and every gridDim.y-th of
// the adapters that its tokens use; its 8 wavefronts split the share and their
// sums are added in LDS in a fixed order.  A's rows are the product's rows,
// tokens its columns: a token keeps the columns of its own adapter only.
// ---------------------------------------------------------------------------
template <class Ad, int RF>
__global__ __launch_bounds__(kThinThreads) void adapter_shrink_kernel(const typename Ad::E* __restrict__ X, int64_t T, int64_t d,
                                                                      int64_t ldx, const typename Ad::E* __restrict__ A,
                                                                      Adapters ad) {
  typedef typename Ad::E E;
  constexpr int kElems = 16 / sizeof(E), kUnit = 4 * kElems, kBatch = RF == 4 ? 4 : 8;
  __shared__ __align__(16) char red[thin_lds_bytes<RF, 1>()];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * 16 + l16;
  const int share = blockIdx.z % ad.parts, r0 = blockIdx.z / ad.parts * 16 * RF;
  int idx[1];
  adapters_of(idx, ad.index, ad.n, t, T);
  // rows past the last token or the rank are read as row 0: their results are dropped
  const E* x = X + (t < T ? t : 0) * ldx;
  // a lane's chunks are neighbours in pairs, so that the lines of 128 bytes are read at once
  auto chunk = [&](int k) { return (k / 2 * 8 + 2 * g + k % 2) * kElems; };
  const int64_t units = (d + 2 * kUnit - 1) / (2 * kUnit), shares = (int64_t)ad.parts * kThinWaves;
  const int64_t per = (units + shares - 1) / shares, first = (share * kThinWaves + wave) * per;
  const int64_t j0 = min(first, units) * 2 * kUnit, j1 = min(min(first + per, units) * 2 * kUnit, d);
  AdapterWalk<1, 16> walk(idx);
  int place = blockIdx.y;
  for (;; --place) {
    const int use = walk.next(idx);
    if (use == INT_MAX) return;
    if (place) continue;
    place = gridDim.y;
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
    float* to = ad.u_parts + (share * T + t) * ad.pitch;
#pragma unroll
    for (int i = 0; i < (RF == 1 ? 2 : RF); ++i) {             // a row is whole thirty-twos
      const int k = r0 + 16 * i + 4 * g;
      if (k >= ad.pitch) continue;
      f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i < RF && k + e < ad.rank) u[e] = acc[i < RF ? i : 0][0][e];
      *reinterpret_cast<f32x4*>(to + k) = u;
    }
  }
}

// ---------------------------------------------------------------------------
// Many tokens, bf16: tiles of 64 ranks by 64 tokens and a share of the
// contraction, on the tile products, once for every adapter of the tile's
// tokens.  Bound by reading X.
// ---------------------------------------------------------------------------
typedef ShapeTile<OpBf16, 0>::T ShrinkTile;
__global__ __launch_bounds__(ShrinkTile::kThreads) void adapter_shrink_tile_kernel(Operand X, const uint16_t* __restrict__ A, int64_t d,
                                                                                   Adapters ad) {
  extern __shared__ __align__(1024) char shrink_lds[];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * 64;
  const int r0 = blockIdx.y * 64, share = blockIdx.z;
  const int kchunks = (int)(d / 8), steps = (kchunks + kStepChunks - 1) / kStepChunks;
  const int per = (steps + 2 * ad.parts - 1) / (2 * ad.parts) * 2, s0 = min(share * per, steps), s1 = min(s0 + per, steps);
  int idx[4];
  adapters_of(idx, ad.index, ad.n, t0 + l16, X.rows);
  AdapterWalk<4, 16> walk(idx);
  for (int use = walk.next(idx); use != INT_MAX; use = walk.next(idx)) {
    const Operand a = {(const char*)(A + (int64_t)use * ad.rank * d), 2 * d, ad.rank, nullptr, 0};
    f32x4 acc[ShrinkTile::TM][ShrinkTile::TN] = {};
    if (s0 < s1) ShrinkTile::run(acc, a, r0, X, t0, kchunks, s0, s1, shrink_lds);
    __syncthreads();                               // nobody reads the operands in LDS any more
#pragma unroll
    for (int j = 0; j < ShrinkTile::TN; ++j) {
      const int64_t t = t0 + wave % 2 * 32 + 16 * j + l16;
      if ((wave % 2 ? idx[2 + j] : idx[j]) != use) continue;
#pragma unroll
      for (int i = 0; i < ShrinkTile::TM; ++i) {
        const int k = r0 + wave / 2 * 32 + 16 * i + 4 * (lane >> 4);
        if (k < ad.pitch) *reinterpret_cast<f32x4*>(ad.u_parts + (share * X.rows + t) * ad.pitch + k) = acc[i][j];
      }
    }
  }
}

// U from its parts as three bf16 numbers, 4 elements a lane
__global__ __launch_bounds__(kBlockThreads) void adapter_round_kernel(Adapters ad, int64_t T) {
  const int quads = ad.pitch / 4;
  for (int64_t i = (int64_t)blockIdx.x * kBlockThreads + threadIdx.x; i < T * quads; i += (int64_t)gridDim.x * kBlockThreads) {
    const int64_t t = i / quads;
    const int k = (int)(i - t * quads) * 4, use = ad.index[t];
    if (use < 0 || use >= ad.n) continue;          // never used
    f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < ad.parts; ++p) u += *reinterpret_cast<const f32x4*>(ad.u_parts + (p * T + t) * ad.pitch + k);
    if (ad.factors) u *= ad.factors[use];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = k + e < ad.rank ? u[e] : 0.0f;
    uint16_t* to = ad.u16 + t * ad.pitch + k;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const uint32_t h0 = pack_bf16x2(u[0], u[1]), h1 = pack_bf16x2(u[2], u[3]);
      *reinterpret_cast<uint2*>(to + n * T * ad.pitch) = make_uint2(h0, h1);
      u[0] -= __uint_as_float(h0 << 16), u[1] -= __uint_as_float(h0 & 0xffff0000u);
      u[2] -= __uint_as_float(h1 << 16), u[3] -= __uint_as_float(h1 & 0xffff0000u);
    }
  }
}

// B with rows of `pitch` elements, filled up with 0: ranks that are not whole
// 16-byte chunks, for the product's tiles.  8 elements a lane.
__global__ __launch_bounds__(kBlockThreads) void adapter_pad_kernel(const uint16_t* __restrict__ B, int64_t rows, int rank, int pitch,
                                                                    uint16_t* __restrict__ padded) {
  const int chunks = pitch / 8;
  for (int64_t i = (int64_t)blockIdx.x * kBlockThreads + threadIdx.x; i < rows * chunks; i += (int64_t)gridDim.x * kBlockThreads) {
    const int64_t row = i / chunks;
    const int k = (int)(i - row * chunks) * 8;
    *reinterpret_cast<i32x4*>(padded + 8 * i) = load_chunk(B + row * rank, k, rank);
  }
}

// ---------------------------------------------------------------------------
// The adapters' part of Y in fp32: a workgroup takes 16 tokens by 32 channels,
// its wavefronts every fourth adapter of these tokens each.  A token has one
// adapter, so one wavefront has all of its row; rows of none are 0.
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 256, kExpandRows = 32;
template <class Ad>
__global__ __launch_bounds__(kExpandThreads) void adapter_expand_kernel(Adapters ad, int64_t T, int64_t N) {
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * kExpandRows;
  for (int64_t t = (int64_t)blockIdx.y * 16 + l16; t - l16 < T; t += (int64_t)gridDim.y * 16) {
    f32x4 acc[2][1] = {};
    const TokenAdapters<1> own(ad, t, T);
    const bool had = add_adapters<Ad, 4>(acc, ad, own, m0 + l16, t, T, N, wave, kExpandThreads / kWave);
    if (t >= T || !(had || (own.idx[0] == INT_MAX && wave == 0))) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (m0 + 16 * i + 4 * g < ad.delta_pitch)
        *reinterpret_cast<f32x4*>(ad.delta + t * ad.delta_pitch + m0 + 16 * i + 4 * g) = acc[i][0];
  }
}

// ===========================================================================
// launchers
// ===========================================================================
static int64_t adapter_pitch(int64_t rank) { return (rank + 31) / 32 * 32; }
static int64_t adapter_delta_pitch(int64_t N) { return (N + 3) / 4 * 4; }
static int64_t rank_tiles(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }
// Shares of the contraction: few tokens leave most CUs idle (T = 1, d = 4096:
// one workgroup 6.8 us), tiles are to be two a CU.
static int adapter_parts(int64_t T, int64_t d, int64_t rank) {
  const int64_t steps = tiles_of(d, 64);
  const int64_t items = T <= 256 ? tiles_of(T, 16) * 16 : tiles_of(T, 64) * tiles_of(rank, 64);
  return (int)std::max<int64_t>(1, std::min<int64_t>({kMostAdapterParts, steps / 16, tiles_of(2 * kCus, items)}));
}
// U's parts, U in bf16, the adapters' part of Y or B filled up
struct AdapterLayout {
  int parts;
  size_t second, third, bytes;
};
static AdapterLayout adapter_layout(int64_t T, int64_t N, int64_t d, int32_t dt, int64_t rank) {
  AdapterLayout p;
  p.parts = adapter_parts(T, d, rank);
  p.second = round_up((size_t)p.parts * T * adapter_pitch(rank) * sizeof(float), 256);
  p.third = p.second + round_up((size_t)T * adapter_pitch(rank) * 6, 256);
  p.bytes = adapters_in_delta(T, N, dt, rank) ? p.third + (size_t)T * adapter_delta_pitch(N) * 4 : p.third;
  return p;
}
size_t adapter_workspace_bytes(int64_t T, int64_t N, int64_t d, int32_t dt, int64_t rank) {
  return adapter_layout(T, N, d, dt, rank).bytes;
}
// workgroups that share the adapters of 16 tokens, up to 16 where there are few tokens
static int64_t adapter_slots(int64_t T, int64_t n) {
  return std::max<int64_t>(1, std::min<int64_t>({n, 16, tiles_of(2 * kCus, tiles_of(T, 16))}));
}
bool adapter_grid_fits(int64_t T, int64_t N, int64_t rank) {
  return grid_holds(tiles_of(T, 16), kThinThreads) && tiles_of(rank, 16 * rank_tiles(rank)) * kMostAdapterParts <= 65535 &&
         grid_holds(tiles_of(N, kExpandRows), kExpandThreads) && tiles_of(T, 16) <= (int64_t(1) << 27);
}

template <class Ad, int RF>
static int shrink_as(const void* X, int64_t T, int64_t d, int64_t ldx, const void* A, const Adapters& ad, hipStream_t st) {
  typedef typename Ad::E E;
  const dim3 grid((unsigned)tiles_of(T, 16), (unsigned)adapter_slots(T, ad.n), (unsigned)(tiles_of(ad.rank, 16 * RF) * ad.parts));
  hipLaunchKernelGGL((adapter_shrink_kernel<Ad, RF>), grid, dim3(kThinThreads), 0, st, (const E*)X, T, d, ldx, (const E*)A, ad);
  return check_launch("adapter_shrink_kernel");
}
template <class Ad>
static int shrink_of(const void* X, int64_t T, int64_t d, int64_t ldx, const void* A, const Adapters& ad, hipStream_t st) {
  const int64_t tiles = rank_tiles(ad.rank);
  if (tiles == 1) return shrink_as<Ad, 1>(X, T, d, ldx, A, ad, st);
  if (tiles == 2) return shrink_as<Ad, 2>(X, T, d, ldx, A, ad, st);
  return shrink_as<Ad, 4>(X, T, d, ldx, A, ad, st);
}
int launch_adapter_shrink(const void* X, int32_t xdt, int64_t T, int64_t N, int64_t d, int64_t ldx, const void* A, void* ws,
                          Adapters* ad, hipStream_t st) {
  const AdapterLayout p = adapter_layout(T, N, d, xdt, ad->rank);
  const bool in_delta = adapters_in_delta(T, N, xdt, ad->rank);
  ad->pitch = (int)adapter_pitch(ad->rank);
  ad->parts = p.parts;
  ad->u_parts = (float*)ws;
  ad->u16 = (uint16_t*)((char*)ws + p.second);
  ad->delta = (float*)((char*)ws + p.third);
  ad->delta_pitch = adapter_delta_pitch(N);
  int rc;
  if (xdt == QAMW_F32) {
    rc = shrink_of<AdaptersF32>(X, T, d, ldx, A, *ad, st);
  } else if (T > 256 && d % 8 == 0 && aligned16(X) && ldx % 8 == 0 && ldx <= kMaxRowBytes / 2) {
    const Operand x = {(const char*)X, 2 * ldx, T, nullptr, 0};
    hipLaunchKernelGGL(adapter_shrink_tile_kernel, dim3((unsigned)tiles_of(T, 64), (unsigned)tiles_of(ad->rank, 64), (unsigned)p.parts),
                       dim3(ShrinkTile::kThreads), ShrinkTile::kLdsBytes, st, x, (const uint16_t*)A, d, *ad);
    rc = check_launch("adapter_shrink_tile_kernel");
  } else {
    rc = shrink_of<AdaptersBf16>(X, T, d, ldx, A, *ad, st);
  }
  // Many tokens and a rank of no whole chunks: where B filled up is smaller than the adapters' part of Y would be, it
  // takes that one's place and the tiles multiply it (4000 x 11008 x 4096, 4 adapters of rank 20).
  const bool pad = in_delta && xdt == QAMW_BF16 && T > 256 && (int64_t)ad->n * ad->pitch <= 2 * T;
  if (!rc && pad) {
    const int64_t rows = (int64_t)ad->n * N;
    hipLaunchKernelGGL(adapter_pad_kernel, dim3((unsigned)std::min<int64_t>(tiles_of(rows * (ad->pitch / 8), kBlockThreads), 1 << 16)),
                       dim3(kBlockThreads), 0, st, (const uint16_t*)ad->B, rows, ad->rank, ad->pitch, (uint16_t*)ad->delta);
    rc = check_launch("adapter_pad_kernel");
  }
  if (rc || (in_delta && !pad) || T <= 256) return rc;
  hipLaunchKernelGGL(adapter_round_kernel, dim3((unsigned)std::min<int64_t>(tiles_of(T * ad->pitch / 4, kBlockThreads), 1 << 16)),
                     dim3(kBlockThreads), 0, st, *ad, T);
  if (pad) ad->B = ad->delta, ad->rank = ad->pitch;            // from here on a rank of whole chunks
  return check_launch("adapter_round_kernel");
}

int launch_adapter_expand(int32_t dt, int64_t T, int64_t N, const Adapters& ad, hipStream_t st) {
  const dim3 grid((unsigned)tiles_of(N, kExpandRows), (unsigned)std::min<int64_t>(tiles_of(T, 16), 65535));
  auto kernel = dt == QAMW_F32 ? adapter_expand_kernel<AdaptersF32> : adapter_expand_kernel<AdaptersBf16x3>;
  hipLaunchKernelGGL(kernel, grid, dim3(kExpandThreads), 0, st, ad, T, N);
  return check_launch("adapter_expand_kernel");
}

}  // namespace qamw
