// Softmax cross entropy of hidden states H [T][d] against a vocabulary head
// W [V][d], and its gradient, without keeping the T x V logits.
//
//     z_tv = <H_t, W_v>,   lse_t = log sum_v exp z_tv,   loss_t = lse_t - z_{t, y_t}
//     G_tv = dloss_t (exp(z_tv - lse_t) - [v = y_t]),   dH = G W,   dW = G^T H
//
// A token whose target lies outside [0, V) is not counted: its loss and its
// gradient are 0, whatever the head holds, and its hidden state, NaN or not,
// reaches nothing else.
//
// Forward: a workgroup forms one tile of logits in registers (vocabulary
// entries are the A operand, so a lane holds several logits of one token) and
// leaves per token the tile's largest logit m and sum of exp(z - m); a second
// kernel joins the tiles in a fixed order.
//
// Gradient: the vocabulary is walked in pieces.  Of a piece the logits are
// formed again and turned into G at once, stored in H's type once as G [T][v]
// and once transposed; dW = G^T H is final for the piece, dH = G W is summed
// over the pieces in fp32.  Every product contracts along the operands' rows,
// which is why H and each piece of W are also laid out transposed.  G is
// rounded to bf16 for bf16 inputs, like H and W themselves: an entry is off by
// up to 2^-8, as much as the rounded gradients that it is summed into, which
// are then off by 0.0019 of their norm (T = 4096, V = 131072) to 0.0025 (few
// tokens) where their own rounding gives 0.0017.  For a few tokens and a large
// head both products run without matrix instructions and transposed copies,
// with G in fp32.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "qamw.h"
#include "qamw_device.h"
#include "qamw_internal.h"
#include "tile_product.h"

namespace qamw {

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

template <class Op> struct Elem;
template <> struct Elem<OpBf16> { typedef uint16_t T; };
template <> struct Elem<OpF32> { typedef float T; };
// whether token t counts (targets NULL: all do)
__device__ __forceinline__ bool counts(const int64_t* targets, int64_t t, int64_t V) {
  return !targets || (targets[t] >= 0 && targets[t] < V);
}
// four consecutive elements, 4-element aligned
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }

// ---------------------------------------------------------------------------
// Tile statistics of the logits: part[tile][t] = (max, sum of exp(z - max)),
// and the target's logit from the one tile that holds it.  Bound by the
// matrix instructions, and by the power they draw: T = 2048, V = 32000, d = 4096
// bf16 takes 420 us in a row of calls, 1.28 PFLOP/s, at 1.9 to 2.0 GHz with
// the matrix instructions busy 60 to 65 % of the time (470 us at the median
// of a traced run); a library product of that size runs at 1.20 PFLOP/s.
// ---------------------------------------------------------------------------
// Of one 16-token column of fragments: lane group l / 16 holds the entries
// 16 i + r past the lane's first one, `left` of them (or more) inside the
// vocabulary, `y` the target's place among them (any other number: not here).
// The result is the same in all four lanes of a token.  Targets and the
// vocabulary's end are rare among tiles, so they are looked for once per
// column, not at every logit.
template <int TM, int TN>
__device__ __forceinline__ float2 column_stats(f32x4 (&acc)[TM][TN], int j, int left, int y, float* zt) {
  if (left < 16 * TM)                                               // not the same in all lanes, but so in few tiles
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * i + r >= left) acc[i][j][r] = -INFINITY;
  if (y >= 0 && y < 16 * TM && y < left && (y & 15) < 4)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (y == 16 * i + r) *zt = acc[i][j][r];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32));
  const float base = m == -INFINITY ? 0.0f : m;                     // a tile of -inf alone sums to 0
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) s += exp_of(acc[i][j][r] - base);
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  return make_float2(m, s);
}
// 64-bit places relative to a lane's first entry, as far as 32 bits matter
__device__ __forceinline__ int near32(int64_t x) { return (int)(x < -1 ? -1 : x > 1 << 20 ? 1 << 20 : x); }

template <class Tl, class Op>
__global__ __launch_bounds__(Tl::kThreads) void ce_stats_kernel(Operand W, Operand H, int kchunks, int tiles_m,
                                                                int tiles_n, const int64_t* __restrict__ targets,
                                                                float2* __restrict__ part, float* __restrict__ zt) {
  extern __shared__ __align__(1024) char tile_lds[];
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * Tl::BM, n0 = (int64_t)tn * Tl::BN;
  f32x4 acc[Tl::TM][Tl::TN] = {};
  Tl::run(acc, W, m0, H, n0, kchunks, 0, (kchunks + kStepChunks - 1) / kStepChunks, tile_lds);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int wm = wave / Tl::WN, wn = wave % Tl::WN;
  const int64_t v0 = m0 + wm * (Tl::BM / Tl::WM) + 4 * (lane >> 4);
  const int tl = wn * (Tl::BN / Tl::WN) + (lane & 15);              // token inside the tile
  float2* red = reinterpret_cast<float2*>(tile_lds);                // [WM][BN]
  __syncthreads();                                                  // the tile's operands are no longer read
#pragma unroll
  for (int j = 0; j < Tl::TN; ++j) {
    const int64_t t = n0 + tl + 16 * j;
    const float2 s = column_stats(acc, j, near32(W.rows - v0), t < H.rows ? near32(targets[t] - v0) : -1, zt + t);
    if (lane < 16) red[wm * Tl::BN + tl + 16 * j] = s;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < Tl::BN; k += Tl::kThreads) {
    float2 a = red[k];
#pragma unroll
    for (int w = 1; w < Tl::WM; ++w) {
      const float2 b = red[w * Tl::BN + k];
      const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.0f : m;
      a = make_float2(m, a.y * exp_of(a.x - base) + b.y * exp_of(b.x - base));
    }
    if (n0 + k < H.rows) part[(int64_t)tm * H.rows + n0 + k] = a;
  }
}

// The same for up to 16 tokens, a tile of kThinRows vocabulary entries: bound
// by reading the head once (T = 1, V = 32000, d = 4096 bf16: 48 us, 5.4 TB/s of
// the 5.9 that a plain read reaches).
constexpr int kThinRows = 16;
template <class Op, int U>
__global__ __launch_bounds__(kThinThreads) void ce_stats_thin_kernel(Operand W, Operand H, int kchunks,
                                                                     const int64_t* __restrict__ targets,
                                                                     float2* __restrict__ part, float* __restrict__ zt) {
  __shared__ __align__(16) char red[thin_lds_bytes<1, 1>()];
  const int64_t m0 = (int64_t)blockIdx.x * kThinRows;
  f32x4 acc[1][1] = {};
  thin_run<Op, U>(acc[0][0], W, m0, H, kchunks);
  thin_sum(acc, red);
  if (threadIdx.x >= kWave) return;
  const int lane = threadIdx.x;
  const int64_t t = lane & 15, v = m0 + 4 * (lane >> 4);
  const float2 s = column_stats(acc, 0, near32(W.rows - v), t < H.rows ? near32(targets[t] - v) : -1, zt + t);
  if (lane < 16 && t < H.rows) part[blockIdx.x * H.rows + t] = s;
}

// Joins the tiles' statistics: TB tokens a workgroup and 256 / TB threads a
// token, thread k taking tiles k, k + 256 / TB, ...; then those in order.
template <int TB>
__global__ __launch_bounds__(256) void ce_finish_kernel(const float2* __restrict__ part, const float* __restrict__ zt,
                                                        const int64_t* __restrict__ targets, int64_t T, int64_t V,
                                                        int tiles, float* __restrict__ loss, float* __restrict__ lse) {
  constexpr int kParts = 256 / TB;
  __shared__ float2 red[kParts][TB];
  const int k = threadIdx.x / TB, i = threadIdx.x % TB;
  const int64_t t = (int64_t)blockIdx.x * TB + i;
  float m = -INFINITY, s = 0.0f;
  if (t < T) {
#pragma unroll 8
    for (int q = k; q < tiles; q += kParts) {
      const float2 p = part[(int64_t)q * T + t];
      const float top = fmaxf(m, p.x), base = top == -INFINITY ? 0.0f : top;
      s = s * exp_of(m - base) + p.y * exp_of(p.x - base);
      m = top;
    }
  }
  red[k][i] = make_float2(m, s);
  // pairs at distance kParts / 2, kParts / 4, ..., 1
#pragma unroll
  for (int h = kParts / 2; h; h >>= 1) {
    __syncthreads();
    if (k < h) {
      const float2 a = red[k][i], b = red[k + h][i];
      const float top = fmaxf(a.x, b.x), base = top == -INFINITY ? 0.0f : top;
      red[k][i] = make_float2(top, a.y * exp_of(a.x - base) + b.y * exp_of(b.x - base));
    }
  }
  if (k == 0 && t < T) {
    const float2 a = red[0][i];
    const float top = a.x == -INFINITY ? 0.0f : a.x, rest = logf(a.y);
    const int64_t y = targets[t];
    lse[t] = top + rest;
    // the largest logit and the target's first: where they are one, a small loss keeps its digits
    loss[t] = (y >= 0 && y < V) ? (top - zt[t]) + rest : 0.0f;
  }
}

// The largest |dloss| of the counted tokens, or 1 where that is 0 or not
// finite.  G is kept relative to it: under a mean loss, whose upstream
// gradients are all the same number, -1 + p is then what is rounded to bf16,
// and not a multiple of an arbitrary factor.  (fp32 inputs go without: unit is
// NULL for them, and 1.)
__global__ __launch_bounds__(1024) void ce_upstream_kernel(const float* __restrict__ dloss,
                                                           const int64_t* __restrict__ targets, int64_t T, int64_t V,
                                                           float* __restrict__ unit) {
  __shared__ float red[16];
  float m = 0.0f;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const int64_t y = targets[t];
    if (y >= 0 && y < V) m = fmaxf(m, fabsf(dloss[t]));
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) m = fmaxf(m, red[i]);
    *unit = m > 0.0f && m < INFINITY ? m : 1.0f;
  }
}

// ---------------------------------------------------------------------------
// G / unit of one piece, in the logits' tiles (T = 4096, 20480 entries, d =
// 4096 bf16: 580 us, 1.18 PFLOP/s, 60 us of it writing G twice): vocabulary
// entries v_first + [0, W.rows).  G [T][vp] and Gt [W.rows][tp]; the columns
// past W.rows (to vp) and past T (to tp) are 0.
// ---------------------------------------------------------------------------
template <class Tl, class Op, class E>
__global__ __launch_bounds__(Tl::kThreads) void ce_softmax_grad_kernel(
    Operand W, Operand H, int kchunks, int tiles_m, int tiles_n, const int64_t* __restrict__ targets, int64_t v_first,
    int64_t V, const float* __restrict__ lse, const float* __restrict__ dloss, const float* __restrict__ unit,
    E* __restrict__ G, int64_t vp, E* __restrict__ Gt, int64_t tp) {                     // Gt may be NULL
  extern __shared__ __align__(1024) char tile_lds[];
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * Tl::BM, n0 = (int64_t)tn * Tl::BN;
  f32x4 acc[Tl::TM][Tl::TN] = {};
  Tl::run(acc, W, m0, H, n0, kchunks, 0, (kchunks + kStepChunks - 1) / kStepChunks, tile_lds);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int64_t v0 = m0 + (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4);
  const int64_t t0 = n0 + (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15);
  __syncthreads();                                                  // the tile's operands are no longer read
#pragma unroll
  for (int j = 0; j < Tl::TN; ++j) {
    const int64_t t = t0 + 16 * j;
    int64_t y = -1;
    float l = 0.0f, g = 0.0f;
    if (t < H.rows) {
      y = targets[t];
      l = lse[t];
      g = unit ? dloss[t] / *unit : dloss[t];
    }
    const bool counted = y >= 0 && y < V;
    const int yl = counted ? near32(y - v_first - v0) : -1, left = near32(W.rows - v0);
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = exp_of(acc[i][j][r] - l) * g;
    // the target and the vocabulary's end, rare among tiles, and tokens that are not counted
    if (yl >= 0 && yl < 16 * Tl::TM && (yl & 15) < 4)
#pragma unroll
      for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (yl == 16 * i + r) acc[i][j][r] = acc[i][j][r] - g;
    if (left < 16 * Tl::TM || !counted)
#pragma unroll
      for (int i = 0; i < Tl::TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * i + r >= left || !counted) acc[i][j][r] = 0.0f;
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i) {
      const f32x4 q = acc[i][j];
      const int64_t v = v0 + 16 * i;
      if constexpr (sizeof(E) == 2) {
        *reinterpret_cast<uint2*>(Tile16<Tl::BM>::at(tile_lds, (int)(t - n0), (int)(v - m0))) =
            make_uint2(pack_bf16x2(q[0], q[1]), pack_bf16x2(q[2], q[3]));
      } else {
        if (t < H.rows && v < vp) store4(G + t * vp + v, q);
        if (Gt && t < tp)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (v + r < W.rows) Gt[(v + r) * tp + t] = q[r];
      }
    }
  }
  if constexpr (sizeof(E) == 2) {
    // 16-bit results go through LDS: rows of G and of Gt in runs of 16 bytes a lane
    __syncthreads();
    tile16_rows<Tl>(tile_lds, [&](int t, int v, u32x4 q) {
      if (n0 + t < H.rows && m0 + v < vp) *reinterpret_cast<u32x4*>(G + (n0 + t) * vp + m0 + v) = q;
    });
    if (!Gt) return;
    for (int k = threadIdx.x; k < Tl::BM / 2 * (Tl::BN / 8); k += Tl::kThreads) {
      // 8 lanes along the tokens, 8 along the vocabulary
      const int cell = k / 64, o = cell % (Tl::BN / 64) * 8 + (k & 7), v = (cell / (Tl::BN / 64) * 8 + (k >> 3 & 7)) * 2;
      if (n0 + 8 * o >= tp || m0 + v >= W.rows) continue;
      u32x4 c0, c1;
      Tile16<Tl::BM>::columns(tile_lds, 8 * o, v, c0, c1);
      E* p = Gt + (m0 + v) * tp + n0 + 8 * o;
      *reinterpret_cast<u32x4*>(p) = c0;
      if (m0 + v + 1 < W.rows) *reinterpret_cast<u32x4*>(p + tp) = c1;
    }
  }
}

// ---------------------------------------------------------------------------
// out[c][r] = in[r][c] for r < R and 0 for R <= r < rp; rows whose target is
// not counted read as 0 (targets NULL: all rows count).  64 x 64 tiles
// through LDS, 16 bytes a lane on both sides: 20480 x 4096 bf16 62 us, 5.4 TB/s.
// ---------------------------------------------------------------------------
template <class E>
__global__ __launch_bounds__(256) void ce_transpose_kernel(const E* __restrict__ in, int64_t pitch, int64_t R, int64_t C,
                                                           E* __restrict__ out, int64_t rp,
                                                           const int64_t* __restrict__ targets, int64_t V) {
  constexpr int kUnit = 16 / sizeof(E);                              // elements per 16 bytes; divides C and rp
  __shared__ __align__(16) char tile[64 * 64 * sizeof(E) + (sizeof(E) == 4 ? 64 * 16 : 0)];
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  auto place = [&](int r, int c) __attribute__((always_inline)) {
    if constexpr (sizeof(E) == 2) return Tile16<64>::at(tile, r, c);
    else return tile + r * (64 * 4 + 16) + c * 4;
  };
  for (int64_t c0 = (int64_t)blockIdx.y * 64; c0 < C; c0 += (int64_t)gridDim.y * 64) {
    __syncthreads();
#pragma unroll
    for (int k = threadIdx.x; k < 64 * 64 / kUnit; k += 256) {
      const int y = k / (64 / kUnit), x = k % (64 / kUnit) * kUnit;
      const int64_t r = r0 + y;
      u32x4 v = {0, 0, 0, 0};
      if (r < R && c0 + x < C && counts(targets, r, V))
        v = *reinterpret_cast<const u32x4*>(in + r * pitch + c0 + x);
      *reinterpret_cast<u32x4*>(place(y, x)) = v;
    }
    __syncthreads();
    if constexpr (sizeof(E) == 2) {
      const int o = threadIdx.x & 7, c = (threadIdx.x >> 3) * 2;
      if (r0 + 8 * o < rp && c0 + c < C) {
        u32x4 a, b;
        Tile16<64>::columns(tile, 8 * o, c, a, b);
        E* p = out + (c0 + c) * rp + r0 + 8 * o;
        *reinterpret_cast<u32x4*>(p) = a;
        *reinterpret_cast<u32x4*>(p + rp) = b;
      }
    } else {
#pragma unroll
      for (int k = threadIdx.x; k < 64 * 16; k += 256) {
        const int x = k % 16 * 4, c = k / 16;
        if (r0 + x >= rp || c0 + c >= C) continue;
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float*>(place(x + i, c));
        *reinterpret_cast<f32x4*>(out + (c0 + c) * rp + r0 + x) = v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// C[n][m] = unit sum_k A[m][k] B[n][k] (unit NULL: 1) over K steps split among
// gridDim.y workgroups: split s writes (or adds to) C + s * split_stride.
// Rows n whose target is not counted are written as 0 (targets NULL: all
// count): their G is 0, but not its product with an infinite or NaN weight.
// 4096 x 20480 x 4096 bf16: 511 us (dW) and 516 us (dH), 1.34 PFLOP/s.
// ---------------------------------------------------------------------------
template <class Tl, class Out>
__global__ __launch_bounds__(Tl::kThreads) void ce_product_kernel(Operand A, Operand B, int kchunks, int tiles_m,
                                                                  int tiles_n, int steps_per_split,
                                                                  const float* __restrict__ unit,
                                                                  const int64_t* __restrict__ targets, int64_t V,
                                                                  Out* __restrict__ C, int64_t ldc,
                                                                  int64_t split_stride, bool add) {
  extern __shared__ __align__(1024) char tile_lds[];
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * Tl::BM, n0 = (int64_t)tn * Tl::BN;
  const int steps = (kchunks + kStepChunks - 1) / kStepChunks;
  const int s0 = min((int)blockIdx.y * steps_per_split, steps), s1 = min(s0 + steps_per_split, steps);
  f32x4 acc[Tl::TM][Tl::TN] = {};
  if (s0 < s1) Tl::run(acc, A, m0, B, n0, kchunks, s0, s1, tile_lds);
  Out* out = C + blockIdx.y * split_stride;
  const float u = unit ? *unit : 1.0f;
  if constexpr (sizeof(Out) == 2) {
    tile16_put<Tl>(tile_lds, acc, [&](f32x4 v) { return make_uint2(pack_bf16x2(v[0] * u, v[1] * u), pack_bf16x2(v[2] * u, v[3] * u)); });
    tile16_rows<Tl>(tile_lds, [&](int n, int m, u32x4 q) {            // A.rows is a multiple of 8
      if (n0 + n >= B.rows || m0 + m >= A.rows) return;
      if (!counts(targets, n0 + n, V)) q = u32x4{0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(out + (n0 + n) * ldc + m0 + m) = q;
    });
    return;
  } else {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
    const int64_t m = m0 + (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4);
    const int64_t n = n0 + (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15);
#pragma unroll
    for (int j = 0; j < Tl::TN; ++j) {
      if (n + 16 * j >= B.rows) continue;
      const bool on = counts(targets, n + 16 * j, V);
#pragma unroll
      for (int i = 0; i < Tl::TM; ++i)
        if (m + 16 * i < A.rows) {
          Out* p = out + (n + 16 * j) * ldc + m + 16 * i;
          acc[i][j] = on ? acc[i][j] * u : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if (add) acc[i][j] += *reinterpret_cast<const f32x4*>(p);
          store4(p, acc[i][j]);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// The two products for a few tokens: bound by reading W and writing dW once,
// with no transposed copies.  A thread owns 16 bytes of columns and walks the
// workgroup's vocabulary entries, whose G lies in LDS.  G is kept in fp32 here,
// also for bf16 inputs: with few terms in the sums its rounding would show.
// ---------------------------------------------------------------------------
template <class E> constexpr int cols_of() { return 16 / sizeof(E); }
template <class E>
__device__ __forceinline__ void unpack_cols(u32x4 v, float (&x)[16 / sizeof(E)]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 2) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(v[i]);
    }
  }
}
constexpr int kThinEntries = 128;                                  // vocabulary entries whose G is in LDS at a time
// g[v][t] = G[t][v0 + v] for v < count, t < T; 0 for T <= t < TT
template <int TT>
__device__ __forceinline__ void stage_g(float (&g)[kThinEntries][TT], const float* G, int64_t vp, int64_t v0, int count, int T) {
  for (int k = threadIdx.x; k < kThinEntries * TT; k += 256) {
    const int t = k / kThinEntries, v = k % kThinEntries;
    g[v][t] = t < T && v < count ? G[t * vp + v0 + v] : 0.0f;
  }
}

// sum[block][t][d] (+)= sum over the block's entries v of G[t][v] W[v][:]
template <class E, int TT>
__global__ __launch_bounds__(256) void ce_dh_thin_kernel(const float* __restrict__ G, int64_t vp, const E* __restrict__ W,
                                                         int64_t ldw, int64_t n, int per_block, int T, int d,
                                                         float* __restrict__ sum, bool add) {
  constexpr int C = cols_of<E>();
  __shared__ __align__(16) float g[kThinEntries][TT];
  const int c = (blockIdx.y * 256 + threadIdx.x) * C;
  const int64_t v0 = min((int64_t)blockIdx.x * per_block, n), v1 = min(v0 + per_block, n);
  float acc[TT][C] = {};
  for (int64_t vb = v0; vb < v1; vb += kThinEntries) {
    const int count = (int)min((int64_t)kThinEntries, v1 - vb);
    __syncthreads();
    stage_g<TT>(g, G, vp, vb, count, T);
    __syncthreads();
    if (c >= d) continue;
    const E* p = W + vb * ldw + c;
    // U rows are multiplied while the next U are on their way; past the end the last row is read, and G is 0
    constexpr int U = 8;
    u32x4 now[U], next[U];
    auto load = [&](u32x4 (&r)[U], int v) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < U; ++k) r[k] = *reinterpret_cast<const u32x4*>(p + (int64_t)min(v + k, count - 1) * ldw);
    };
    load(now, 0);
    for (int v = 0; v < count; v += U) {
      load(next, v + U);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float w[C];
        unpack_cols<E>(now[k], w);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < C; ++i) acc[t][i] = fmaf(g[v + k][t], w[i], acc[t][i]);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) now[k] = next[k];
    }
  }
  if (c >= d) return;
#pragma unroll
  for (int t = 0; t < TT; ++t)
    if (t < T) {
      float* p = sum + ((int64_t)blockIdx.x * T + t) * d + c;
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        f32x4 a = {acc[t][i], acc[t][i + 1], acc[t][i + 2], acc[t][i + 3]};
        if (add) a += *reinterpret_cast<const f32x4*>(p + i);
        *reinterpret_cast<f32x4*>(p + i) = a;
      }
    }
}

// dW[v][:] = unit sum_t G[t][v] H[t][:], the counted tokens t
template <class E, int TT>
__global__ __launch_bounds__(256) void ce_dw_thin_kernel(const float* __restrict__ G, int64_t vp, const E* __restrict__ H,
                                                         int64_t ldh, const int64_t* __restrict__ targets, int64_t V,
                                                         int64_t n, int per_block, int T, int d,
                                                         const float* __restrict__ unit, E* __restrict__ dW, int64_t lddw) {
  constexpr int C = cols_of<E>();
  __shared__ __align__(16) float g[kThinEntries][TT];
  const int c = (blockIdx.y * 256 + threadIdx.x) * C;
  const int64_t v0 = (int64_t)blockIdx.x * per_block;               // per_block <= kThinEntries
  const int count = (int)min((int64_t)per_block, n - v0);
  stage_g<TT>(g, G, vp, v0, count, T);
  __syncthreads();
  if (c >= d) return;
  const float u = unit ? *unit : 1.0f;
  float h[TT][C];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t y = t < T ? targets[t] : -1;
    if (y >= 0 && y < V) {
      unpack_cols<E>(*reinterpret_cast<const u32x4*>(H + t * ldh + c), h[t]);
#pragma unroll
      for (int i = 0; i < C; ++i) h[t][i] *= u;
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) h[t][i] = 0.0f;
    }
  }
  E* p = dW + v0 * lddw + c;
  for (int v = 0; v < count; ++v, p += lddw) {
    float a[C] = {};
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < C; ++i) a[i] = fmaf(g[v][t], h[t][i], a[i]);
    if constexpr (sizeof(E) == 2)
      *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                                           pack_bf16x2(a[6], a[7])};
    else
      *reinterpret_cast<f32x4*>(p) = f32x4{a[0], a[1], a[2], a[3]};
  }
}

// dH = unit times many fp32 sums, 16 threads an element: thread k adds sums k,
// k + 16, ..., then the 16 in order; rounded once.  0 for a token that is not
// counted (its sums are not, where a weight is infinite or NaN).
template <class E>
__global__ __launch_bounds__(256) void ce_sum_blocks_kernel(const float* __restrict__ part, int blocks, int64_t stride,
                                                            int64_t T, int d, const float* __restrict__ unit,
                                                            const int64_t* __restrict__ targets, int64_t V,
                                                            E* __restrict__ out, int64_t ldo) {
  __shared__ f32x4 red[16][16];
  const int i = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int64_t per = d / 4, n = T * per, e = (int64_t)blockIdx.x * 16 + i;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (e < n)
#pragma unroll 8
    for (int q = k; q < blocks; q += 16) s += *reinterpret_cast<const f32x4*>(part + q * stride + 4 * e);
  red[k][i] = s;
  __syncthreads();
  if (k || e >= n) return;
#pragma unroll
  for (int q = 1; q < 16; ++q) s += red[q][i];
  if (!counts(targets, e / per, V)) s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  store4(out + e / per * ldo + e % per * 4, unit ? s * *unit : s);
}

// dH = unit times the fp32 sums of the splits, in order, rounded once; 0 for a
// token that is not counted
template <class E>
__global__ __launch_bounds__(256) void ce_sum_splits_kernel(const float* __restrict__ part, int splits, int64_t stride,
                                                            int64_t T, int d, const float* __restrict__ unit,
                                                            const int64_t* __restrict__ targets, int64_t V,
                                                            E* __restrict__ out, int64_t ldo) {
  const float u = unit ? *unit : 1.0f;
  const int64_t per = d / 4, n = T * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    f32x4 s = reinterpret_cast<const f32x4*>(part)[i];
    for (int k = 1; k < splits; ++k) s += *reinterpret_cast<const f32x4*>(part + k * stride + 4 * i);
    if (!counts(targets, i / per, V)) s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    store4(out + i / per * ldo + i % per * 4, s * u);
  }
}

template <class E>
__global__ __launch_bounds__(256) void ce_zero_kernel(E* __restrict__ out, int64_t rows, int d, int64_t ldo) {
  const int64_t per = d / 4, n = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    store4(out + i / per * ldo + i % per * 4, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
}

// ===========================================================================
// launchers
// ===========================================================================
static unsigned blocks_for(int64_t n, int per) { return (unsigned)std::min<int64_t>((n + per - 1) / per, 65536); }

// Up to this many tokens the loss reads the head in thin tiles of 16 entries
// (V = 32000, d = 4096, bf16: T = 1 56.9 us, T = 4 60.0 us; with 64 entries 62.7
// us at T = 1, in 64 x 64 tiles 58.2 us at T = 20).
constexpr int64_t kThinTokens = 4;

static ProductType product_type(int es) { return es == 4 ? kProductF32 : kProductBf16; }
static int64_t steps_of(int64_t elements, int es) { return tiles_of(elements * es, kStepBytes); }
// tile shape of the logits, and its vocabulary entries
static int logits_shape(int64_t T, int64_t V, int d, int es) { return product_plan(product_type(es), V, T, steps_of(d, es), 1).shape; }
static int logits_tile(int64_t T, int64_t V, int d, int es) {
  return T <= kThinTokens ? kThinRows : kShapeTile[logits_shape(T, V, d, es)];
}
bool ce_grid_fits(int64_t T, int64_t V, int d, int32_t dt) {
  if (T <= kThinTokens) return grid_holds(tiles_of(V, kThinRows), kThinThreads);
  const int shape = logits_shape(T, V, d, elem_size(dt));
  return grid_holds(shape_tiles(shape, V, T), shape_threads(shape));
}
size_t ce_workspace_bytes(int64_t T, int64_t V, int d, int32_t dt) {
  return round_up((size_t)tiles_of(V, logits_tile(T, V, d, elem_size(dt))) * T * sizeof(float2), 256) +
         round_up((size_t)T * sizeof(float), 256);
}

static int ce_finish(const float2* part, const float* zt, const int64_t* targets, int64_t T, int64_t V, int tiles, float* loss,
                     float* lse, hipStream_t st) {
  if (T <= 64)
    hipLaunchKernelGGL(ce_finish_kernel<1>, dim3((unsigned)T), dim3(256), 0, st, part, zt, targets, T, V, tiles, loss, lse);
  else
    hipLaunchKernelGGL(ce_finish_kernel<16>, dim3((unsigned)((T + 15) / 16)), dim3(256), 0, st, part, zt, targets, T, V,
                       tiles, loss, lse);
  return check_launch("ce_finish_kernel");
}
template <class Op, class Tl>
static int ce_tiled(const Operand& W, const Operand& H, int kchunks, const int64_t* targets, float* loss, float* lse,
                    void* ws, hipStream_t st) {
  const int tm = (int)tiles_of(W.rows, Tl::BM), tn = (int)tiles_of(H.rows, Tl::BN);
  const int64_t T = H.rows;
  float2* part = (float2*)ws;
  float* zt = (float*)((char*)ws + round_up((size_t)tm * T * sizeof(float2), 256));
  auto kernel = ce_stats_kernel<Tl, Op>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(Tl::kThreads), Tl::kLdsBytes, st, W, H, kchunks, tm, tn,
                     targets, part, zt);
  const int rc = check_launch("ce_stats_kernel");
  return rc ? rc : ce_finish(part, zt, targets, T, W.rows, tm, loss, lse, st);
}
template <class Op>
static int ce_thin(const Operand& W, const Operand& H, int kchunks, const int64_t* targets, float* loss, float* lse, void* ws,
                   hipStream_t st) {
  const int tm = (int)tiles_of(W.rows, kThinRows);
  const int64_t T = H.rows;
  float2* part = (float2*)ws;
  float* zt = (float*)((char*)ws + round_up((size_t)tm * T * sizeof(float2), 256));
  hipLaunchKernelGGL((ce_stats_thin_kernel<Op, 4>), dim3((unsigned)tm), dim3(kThinThreads), 0, st, W, H, kchunks,
                     targets, part, zt);
  const int rc = check_launch("ce_stats_thin_kernel");
  return rc ? rc : ce_finish(part, zt, targets, T, W.rows, tm, loss, lse, st);
}
template <class Op>
static int ce_as(const void* H, int64_t T, int d, int64_t ldh, const void* W, int64_t V, int64_t ldw,
                 const int64_t* targets, float* loss, float* lse, void* ws, hipStream_t st) {
  const int es = sizeof(typename Elem<Op>::T), kchunks = d / Op::kElems;
  const Operand a = {(const char*)W, ldw * es, V, nullptr, 0}, b = {(const char*)H, ldh * es, T, nullptr, 0};
  if (T <= kThinTokens) return ce_thin<Op>(a, b, kchunks, targets, loss, lse, ws, st);
  return with_shape<Op>(logits_shape(T, V, d, es),
                        [&](auto tile) { return ce_tiled<Op, decltype(tile)>(a, b, kchunks, targets, loss, lse, ws, st); });
}
int launch_cross_entropy(const void* H, int32_t dt, int64_t T, int d, int64_t ldh, const void* W, int64_t V, int64_t ldw,
                         const int64_t* targets, float* loss, float* lse, void* ws, hipStream_t st) {
  return dt == QAMW_F32 ? ce_as<OpF32>(H, T, d, ldh, W, V, ldw, targets, loss, lse, ws, st)
                        : ce_as<OpBf16>(H, T, d, ldh, W, V, ldw, targets, loss, lse, ws, st);
}

constexpr int64_t kPieceTile = kShapeTile[kShapes - 1];
// G, Gt and Wt of one piece.  More of it means fewer launches, each with a
// last round of workgroups that fills the CUs badly: T = 4096, V = 131072,
// d = 4096 takes 15.1 ms at 128 MiB, 14.7 ms at 420 MiB and 14.5 ms at
// 820 MiB.
constexpr int64_t kCeBudget = (int64_t)512 << 20;

// Whether the products run without transposed copies and matrix instructions
// (and with G in fp32): for up to 4 tokens, and up to 16 with a head of some
// size, whose copies would cost more than all else (loss and gradient at V =
// 32000, d = 4096, bf16: T = 1 214 us against 356 us, T = 16 302 us, T = 17 361
// us; V = 5003, d = 512: fp32, 10 MB, T = 16 57 us, T = 17 66 us, but bf16, 5
// MB, 50 us and 42 us).  The limit is one of time: beyond it bf16's G is
// rounded however few the tokens are, and dH and dW are off by up to 0.0025 of
// their norm where their own rounding alone gives 0.0017.
static bool thin_gradient(int64_t T, int64_t V, int d, int es) {
  return T <= kThinTokens || (T <= 16 && V * d * es >= (int64_t(8) << 20));
}

// Sizes and places of the gradient's workspace.
struct CeGradPlan {
  int64_t piece;            // vocabulary entries per piece
  int64_t vp, tp;           // row pitches of G and Wt, of Gt and Ht (elements)
  bool thin;                // a few tokens: no transposed copies
  int blocks;               // thin: vocabulary blocks of a piece, each with an fp32 sum of dH
  ProductPlan dh;           // dH's product over one piece: splits hold fp32 sums of their own over all pieces
  size_t unit, g, gt, wt, ht, sum, bytes;
};
static CeGradPlan ce_grad_plan(int64_t T, int64_t V, int d, int es) {
  CeGradPlan p;
  // Entries whose G, Gt and Wt fit the budget, as whole rounds of large tiles
  // over the CUs where a round is no more than that (T = 4096: 16 tiles of
  // tokens by 16 of vocabulary), then evened out over the pieces.
  const int64_t budget = kCeBudget;
  int64_t fit = std::min<int64_t>(budget / ((2 * T + d) * es), kMaxRowBytes / es) / kPieceTile;   // tiles
  fit = std::max<int64_t>(fit, 1);
  int64_t round = kCus;
  for (int64_t tn = tiles_of(T, kPieceTile); round > 1 && tn % 2 == 0; tn /= 2) round /= 2;
  if (round <= fit) fit = fit / round * round;
  else round = 1;
  const int64_t all = tiles_of(V, kPieceTile), pieces = tiles_of(all, fit);
  p.piece = std::min<int64_t>(tiles_of(tiles_of(all, pieces), round) * round * kPieceTile, (V + 7) / 8 * 8);
  p.vp = p.piece;
  p.tp = (T + 7) / 8 * 8;
  p.dh = product_plan(product_type(es), d, T, steps_of(p.vp, es), 16);
  p.thin = thin_gradient(T, V, d, es);
  // enough blocks for two workgroups a CU, of at least 32 entries
  p.blocks = (int)std::min<int64_t>(tiles_of(p.piece, 32), tiles_of(2 * kCus, tiles_of((int64_t)d * es, 4096)));
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at += round_up(bytes, 256); return o; };
  p.unit = take(sizeof(float));
  p.g = take((size_t)T * p.vp * (p.thin ? sizeof(float) : es));
  p.gt = p.wt = p.ht = 0;
  if (!p.thin) {
    p.gt = take((size_t)p.piece * p.tp * es);
    p.wt = take((size_t)d * p.vp * es);
    p.ht = take((size_t)d * p.tp * es);
  }
  p.sum = take((size_t)(p.thin ? p.blocks : p.dh.splits) * T * d * sizeof(float));
  p.bytes = at;
  return p;
}
size_t ce_grad_workspace_bytes(int64_t T, int64_t V, int d, int32_t dt) { return ce_grad_plan(T, V, d, elem_size(dt)).bytes; }

template <class Op, class Tl, class E>
static int softmax_grad_tiled(const Operand& W, const Operand& H, int kchunks, const int64_t* targets, int64_t v0, int64_t V,
                              const float* lse, const float* dloss, const float* unit, E* G, int64_t vp, E* Gt, int64_t tp,
                              hipStream_t st) {
  const int tm = (int)tiles_of(W.rows, Tl::BM), tn = (int)tiles_of(H.rows, Tl::BN);
  auto kernel = ce_softmax_grad_kernel<Tl, Op, E>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn)), dim3(Tl::kThreads), Tl::kLdsBytes, st, W, H, kchunks, tm, tn,
                     targets, v0, V, lse, dloss, unit, G, vp, Gt, tp);
  return check_launch("ce_softmax_grad_kernel");
}
template <class Tl, class Out>
static int product_tiled(const Operand& A, const Operand& B, int kchunks, int splits, const float* unit,
                         const int64_t* targets, int64_t V, Out* C, int64_t ldc, int64_t split_stride, bool add,
                         hipStream_t st) {
  const int tm = (int)tiles_of(A.rows, Tl::BM), tn = (int)tiles_of(B.rows, Tl::BN);
  const int steps = (kchunks + kStepChunks - 1) / kStepChunks, per = (steps + splits - 1) / splits;
  auto kernel = ce_product_kernel<Tl, Out>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tm * tn), (unsigned)splits), dim3(Tl::kThreads), Tl::kLdsBytes, st, A, B,
                     kchunks, tm, tn, per, unit, targets, V, C, ldc, split_stride, add);
  return check_launch("ce_product_kernel");
}
template <class Op, class Out>
static int product(const Operand& A, const Operand& B, int kchunks, const ProductPlan& p, const float* unit,
                   const int64_t* targets, int64_t V, Out* C, int64_t ldc, int64_t split_stride, bool add, hipStream_t st) {
  return with_shape<Op>(p.shape, [&](auto tile) {
    return product_tiled<decltype(tile), Out>(A, B, kchunks, p.splits, unit, targets, V, C, ldc, split_stride, add, st);
  });
}

// f(std::integral_constant) with the smallest of 1, 4 and 16 that holds T
template <class F>
static int with_tokens(int64_t T, F&& f) {
  if (T == 1) return f(std::integral_constant<int, 1>());
  if (T <= 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 16>());
}
template <class E>
static int dh_thin(const float* G, int64_t vp, const E* W, int64_t ldw, int64_t n, int blocks, int64_t T, int d, float* sum, bool add,
                   hipStream_t st) {
  return with_tokens(T, [&](auto tt) {
    auto kernel = ce_dh_thin_kernel<E, decltype(tt)::value>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks, (unsigned)tiles_of(d, 256 * cols_of<E>())), dim3(256), 0, st, G, vp, W, ldw,
                       n, (int)tiles_of(n, blocks), (int)T, d, sum, add);
    return check_launch("ce_dh_thin_kernel");
  });
}
template <class E>
static int dw_thin(const float* G, int64_t vp, const E* H, int64_t ldh, const int64_t* targets, int64_t V, int64_t n, int64_t T, int d,
                   const float* unit, E* dW, int64_t lddw, hipStream_t st) {
  return with_tokens(T, [&](auto tt) {
    auto kernel = ce_dw_thin_kernel<E, decltype(tt)::value>;
    // four workgroups a CU, of 8 to kThinEntries entries
    const int64_t across = tiles_of(d, 256 * cols_of<E>());
    const int per = (int)std::min<int64_t>(std::max<int64_t>(n * across / (4 * kCus), 8), kThinEntries);
    hipLaunchKernelGGL(kernel, dim3((unsigned)tiles_of(n, per), (unsigned)across), dim3(256), 0, st, G, vp, H, ldh, targets, V, n,
                       per, (int)T, d, unit, dW, lddw);
    return check_launch("ce_dw_thin_kernel");
  });
}

template <class Op>
static int ce_grad_as(const void* H, int64_t T, int d, int64_t ldh, const void* W, int64_t V, int64_t ldw,
                      const int64_t* targets, const float* lse, const float* dloss, void* dH, int64_t lddh, void* dW,
                      int64_t lddw, void* ws, hipStream_t st) {
  typedef typename Elem<Op>::T E;
  const int es = sizeof(E);
  const CeGradPlan p = ce_grad_plan(T, V, d, es);
  char* w = (char*)ws;
  E *G = (E*)(w + p.g), *Gt = (E*)(w + p.gt), *Wt = (E*)(w + p.wt), *Ht = (E*)(w + p.ht);
  float *unit = (float*)(w + p.unit), *sum = (float*)(w + p.sum);
  const int64_t split_stride = T * (int64_t)d;
  const unsigned dtiles = (unsigned)std::min<int64_t>((d + 63) / 64, 65535);
  int rc;
  if (es == 2) {
    hipLaunchKernelGGL(ce_upstream_kernel, dim3(1), dim3(1024), 0, st, dloss, targets, T, V, unit);
    if ((rc = check_launch("ce_upstream_kernel"))) return rc;
  } else {
    unit = nullptr;
  }
  E* const Gt_out = dW && !p.thin ? Gt : nullptr;
  if (dW && !p.thin) {
    hipLaunchKernelGGL((ce_transpose_kernel<E>), dim3((unsigned)((p.tp + 63) / 64), dtiles), dim3(256), 0, st,
                       (const E*)H, ldh, T, (int64_t)d, Ht, p.tp, targets, V);
    if ((rc = check_launch("ce_transpose_kernel"))) return rc;
  }
  for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
    const int64_t n = std::min<int64_t>(p.piece, V - v0);
    const Operand Wp = {(const char*)W + v0 * ldw * es, ldw * es, n, nullptr, 0};
    const Operand Hp = {(const char*)H, ldh * es, T, nullptr, 0};
    const int kd = d / Op::kElems;
    const int shape = logits_shape(T, n, d, es);
    if (p.thin) {                                                   // so few tokens take the smallest tiles
      float* G32 = (float*)G;
      auto grad = [&](auto tile) {
        return softmax_grad_tiled<Op, decltype(tile), float>(Wp, Hp, kd, targets, v0, V, lse, dloss, unit, G32, p.vp, nullptr, 0, st);
      };
      if constexpr (std::is_same<Op, OpF32>::value) rc = grad(typename ShapeTile<Op, 1>::T());
      else rc = shape ? grad(typename ShapeTile<Op, 1>::T()) : grad(typename ShapeTile<Op, 0>::T());
      if (rc) return rc;
      if (dW && (rc = dw_thin<E>(G32, p.vp, (const E*)H, ldh, targets, V, n, T, d, unit, (E*)dW + v0 * lddw, lddw, st))) return rc;
      if (dH && (rc = dh_thin<E>(G32, p.vp, (const E*)W + v0 * ldw, ldw, n, p.blocks, T, d, sum, v0 > 0, st))) return rc;
      continue;
    }
    rc = with_shape<Op>(shape, [&](auto tile) {
      return softmax_grad_tiled<Op, decltype(tile), E>(Wp, Hp, kd, targets, v0, V, lse, dloss, unit, G, p.vp, Gt_out, p.tp, st);
    });
    if (rc) return rc;
    if (dW) {
      const Operand a = {(const char*)Ht, p.tp * es, d, nullptr, 0}, b = {(const char*)Gt, p.tp * es, n, nullptr, 0};
      const ProductPlan whole = product_plan(product_type(es), d, n, steps_of(p.tp, es), 1);
      if ((rc = product<Op, E>(a, b, (int)(p.tp / Op::kElems), whole, unit, nullptr, V, (E*)dW + v0 * lddw, lddw, 0, false, st)))
        return rc;
    }
    if (dH) {
      const int64_t np = (n + 7) / 8 * 8;                           // whole chunks; G and Wt hold 0 past n
      hipLaunchKernelGGL((ce_transpose_kernel<E>), dim3((unsigned)((np + 63) / 64), dtiles), dim3(256), 0, st,
                         (const E*)W + v0 * ldw, ldw, n, (int64_t)d, Wt, p.vp, (const int64_t*)nullptr, V);
      if ((rc = check_launch("ce_transpose_kernel"))) return rc;
      const Operand a = {(const char*)Wt, p.vp * es, d, nullptr, 0}, b = {(const char*)G, p.vp * es, T, nullptr, 0};
      const int kc = (int)(np / Op::kElems);
      if (n == V && p.dh.splits == 1)                               // one piece, one sum: the result itself
        return product<Op, E>(a, b, kc, p.dh, unit, targets, V, (E*)dH, lddh, 0, false, st);
      if ((rc = product<Op, float>(a, b, kc, p.dh, nullptr, nullptr, V, sum, d, split_stride, v0 > 0, st))) return rc;
    }
  }
  if (!dH) return QAMW_OK;
  if (p.thin) {
    hipLaunchKernelGGL((ce_sum_blocks_kernel<E>), dim3((unsigned)tiles_of(T * (d / 4), 16)), dim3(256), 0, st, sum, p.blocks,
                       split_stride, T, d, unit, targets, V, (E*)dH, lddh);
    return check_launch("ce_sum_blocks_kernel");
  }
  hipLaunchKernelGGL((ce_sum_splits_kernel<E>), dim3(blocks_for(T * (d / 4), 256)), dim3(256), 0, st, sum, p.dh.splits,
                     split_stride, T, d, unit, targets, V, (E*)dH, lddh);
  return check_launch("ce_sum_splits_kernel");
}
int launch_cross_entropy_grad(const void* H, int32_t dt, int64_t T, int d, int64_t ldh, const void* W, int64_t V,
                              int64_t ldw, const int64_t* targets, const float* lse, const float* dloss, void* dH,
                              int64_t lddh, void* dW, int64_t lddw, void* ws, hipStream_t st) {
  return dt == QAMW_F32
             ? ce_grad_as<OpF32>(H, T, d, ldh, W, V, ldw, targets, lse, dloss, dH, lddh, dW, lddw, ws, st)
             : ce_grad_as<OpBf16>(H, T, d, ldh, W, V, ldw, targets, lse, dloss, dH, lddh, dW, lddw, ws, st);
}
// the gradient of no tokens
int launch_zero_rows(void* out, int32_t dt, int64_t rows, int d, int64_t ldo, hipStream_t st) {
  const dim3 grid(blocks_for(rows * (d / 4), 256)), block(256);
  if (dt == QAMW_F32) hipLaunchKernelGGL((ce_zero_kernel<float>), grid, block, 0, st, (float*)out, rows, d, ldo);
  else hipLaunchKernelGGL((ce_zero_kernel<uint16_t>), grid, block, 0, st, (uint16_t*)out, rows, d, ldo);
  return check_launch("ce_zero_kernel");
}

}  // namespace qamw
