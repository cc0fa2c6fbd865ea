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
#include <type_traits>

#include "qamw.h"
#include "mx4_adapter.h"
#include "mx4_device.h"
#include "qamw_device.h"
#include "qamw_internal.h"
#include "tile_product.h"

namespace qamw {

// 32 consecutive 16-bit elements as one lane holds them.
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <class Mem> struct RawBlock;
template <bool kBf16>
struct RawBlock16 {
  i32x4 r[4];
  __device__ __forceinline__ uint32_t max_bits() const {
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, r[i / 4][i % 4] & 0x7fff7fff));
    const uint16_t h = m[0] > m[1] ? m[0] : m[1];
    return kBf16 ? (uint32_t)h << 16 : __float_as_uint((float)__builtin_bit_cast(_Float16, h));
  }
  __device__ __forceinline__ i32x4 encode(uint32_t code) const {
    if (code == 255u) return i32x4{0, 0, 0, 0};
    const float s = __uint_as_float(code << 23);
    i32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c = 0;
      if constexpr (kBf16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (int)r[i][0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (int)r[i][1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (int)r[i][2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, (int)r[i][3]), s, 3);
      } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, (int)r[i][0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, (int)r[i][1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, (int)r[i][2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, (int)r[i][3]), s, 3);
      }
      out[i] = (int)c;
    }
    return out;
  }
};
template <> struct RawBlock<MemBf16> : RawBlock16<true> {};
template <> struct RawBlock<MemF16> : RawBlock16<false> {};
// ---------------------------------------------------------------------------
// Quantisation: a lane holds 8 elements, a quad of lanes a block, whose
// largest exponent two lane exchanges give.  Bound by memory: every element is
// read once and its half byte (and its value) written once.  4096 x 11008
// bf16 with values: 35 us, 204 MB, 5.8 TB/s.  A workgroup is blockDim.x lanes
// along a row by blockDim.y rows.
// ---------------------------------------------------------------------------
template <class In, class Val, int kGroups>
__global__ __launch_bounds__(kBlockThreads) void mx4_quantize_kernel(
    const typename In::T* __restrict__ W, int64_t N, int d, int64_t ldw, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales, int nb, int scale_pitch, typename Val::T* __restrict__ values, int64_t ldv) {
  const int per_row = 4 * nb;                                             // groups of 8 in a row
  const int u0 = blockIdx.x * blockDim.x * kGroups + threadIdx.x;
  for (int64_t n = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; n < N; n += (int64_t)gridDim.y * blockDim.y) {
    float x[kGroups][8];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int u = u0 + k * blockDim.x;                                  // whole quads are in or out
      if (u < per_row) load8<In>(W + n * ldw, 8 * u, d, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int u = u0 + k * blockDim.x;
      if (u >= per_row) continue;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[k][i]) & 0x7fffffffu);
      const uint32_t code = scale_code(quad_max(m));
      const uint32_t c = encode8(x[k], code);
      *reinterpret_cast<uint32_t*>(codes + n * (int64_t)nb * 16 + 4 * u) = c;
      uint8_t* srow = scales + n * scale_pitch;
      if ((u & 3) == 0) {
        srow[u >> 2] = (uint8_t)code;
        if (u == per_row - 4)
          for (int q = nb; q < scale_pitch; ++q) srow[q] = 0;
      }
      if (values) {
        decode8(c, code, x[k]);
        store8<Val>(values + n * ldv, 8 * u, d, x[k]);
      }
    }
  }
}

// The values of 8 elements a lane.  Bound by memory: 11008 x 4096 to bf16 19
// us, 114 MB, 6.0 TB/s.
template <class Out>
__global__ __launch_bounds__(kBlockThreads) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                       const uint8_t* __restrict__ scales, int64_t N,
                                                                       int d, int nb, int scale_pitch,
                                                                       typename Out::T* __restrict__ W, int64_t ldo) {
  const int per_row = 4 * nb;
  for (int64_t n = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; n < N; n += (int64_t)gridDim.y * blockDim.y) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= per_row) continue;
    float x[8];
    decode8(*reinterpret_cast<const uint32_t*>(codes + n * (int64_t)nb * 16 + 4 * u), scales[n * scale_pitch + (u >> 2)], x);
    store8<Out>(W + n * ldo, 8 * u, d, x);
  }
}

// ---------------------------------------------------------------------------
// Y[t][n] = sum_k X^[t][k] W^[n][k] on v_mfma_scale_f32_16x16x128: the
// instruction multiplies 128 four-bit products per result and applies both
// blocks' scales, so nothing is decoded.  Weights are the A operand: a lane
// then holds 4 consecutive channels n of one token.  T = 8192, 11008 x 4096: 231
// us, 3.2 PFLOP/s, in a row of calls (251 us with the quantisation of X).  The
// clock stays near its highest (2.27 of 2.4 GHz), so power does not bound it:
// a K step of a 256 x 256 tile takes about 4300 cycles, in which the matrix
// instructions are busy for 2050.  Over the whole launch they are busy 32 % of
// the time and LDS reads 21 %: neither is full, and wavefronts wait for 28 % of
// their cycles and to issue for 43 %.  With 16 K steps a tile's first loads and
// its stores add 4 steps' time, and of the sixth round of tiles 0.4 is used.
// Rows of 13824: 3.9 PFLOP/s, 46 % busy at 2.04 GHz (the instructions alone, on
// registers, reach 6.8).  This tile has all 256 registers and one too few: the
// compiler spills one, 8 bytes a lane.
// ---------------------------------------------------------------------------
// Workgroups below `whole` take one tile each; those after it take a share of
// K of a tile, `splits` to a tile, and leave fp32 results in
// part[tile - whole][split][BN][BM] for mx4_sum_tail_kernel.  Adapters are
// added by the workgroup that holds a tile's first share.
template <class Tl, class Out, class Ad>
__global__ __launch_bounds__(Tl::kThreads) void mx4_matmul_kernel(Operand W, Operand X, int kchunks, int tiles_m,
                                                                  int tiles_n, int whole, int splits,
                                                                  typename Out::T* __restrict__ Y, int64_t ldy,
                                                                  float* __restrict__ part, Adapters ad) {
  extern __shared__ __align__(1024) char tile_lds[];
  const int id = blockIdx.x, steps = (kchunks + kStepChunks - 1) / kStepChunks;
  const bool split = id >= whole;
  int tm, tn, s0 = 0, s1 = steps;
  if (split) {
    tile_at(whole + (id - whole) / splits, tiles_m, tiles_n, tm, tn);
    // an even number of steps each: scale codes are copied for two steps at a time
    const int per = (steps + 2 * splits - 1) / (2 * splits) * 2;
    s0 = min((id - whole) % splits * per, steps);
    s1 = min(s0 + per, steps);
  } else {
    tile_at(xcd_place(id, whole), tiles_m, tiles_n, tm, tn);
  }
  const int64_t m0 = (int64_t)tm * Tl::BM, n0 = (int64_t)tn * Tl::BN;
  f32x4 acc[Tl::TM][Tl::TN] = {};
  if constexpr (Ad::kDelta)
    if (s0 == 0) {
      const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
      load_delta(acc, ad, m0 + (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4),
                 n0 + (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15), X.rows);
    }
  if (s0 < s1) Tl::run(acc, W, m0, X, n0, kchunks, s0, s1, tile_lds);
  if constexpr (Ad::kOn)
    if (s0 == 0) add_adapters_tile<Ad, Tl>(acc, ad, m0, n0, X.rows, W.rows, tile_lds);
  if (!split) {
    store_tile<Tl, Out>(Y, ldy, n0, X.rows, m0, W.rows, acc, tile_lds);
    return;
  }
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int ml = (wave / Tl::WN) * (Tl::BM / Tl::WM) + 4 * (lane >> 4), tl = (wave % Tl::WN) * (Tl::BN / Tl::WN) + (lane & 15);
  float* p = part + ((int64_t)(id - whole) * Tl::BN + tl) * Tl::BM + ml;
#pragma unroll
  for (int j = 0; j < Tl::TN; ++j)
#pragma unroll
    for (int i = 0; i < Tl::TM; ++i) *reinterpret_cast<f32x4*>(p + 16 * j * Tl::BM + 16 * i) = acc[i][j];
}

// Y of the split tiles: a tile per blockIdx.y, its shares added in order
template <class Tl, class Out>
__global__ __launch_bounds__(256) void mx4_sum_tail_kernel(const float* __restrict__ part, int whole, int splits, int tiles_m,
                                                           int tiles_n, int64_t T, int64_t N,
                                                           typename Out::T* __restrict__ Y, int64_t ldy) {
  int tm, tn;
  tile_at(whole + (int)blockIdx.y, tiles_m, tiles_n, tm, tn);
  const int e = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4, m = e % Tl::BM, n = e / Tl::BM;
  const int64_t t = (int64_t)tn * Tl::BN + n, c = (int64_t)tm * Tl::BM + m;
  if (t >= T || c >= N) return;
  const float* p = part + (int64_t)blockIdx.y * splits * (Tl::BM * Tl::BN) + e;
  f32x4 s = *reinterpret_cast<const f32x4*>(p);
  for (int k = 1; k < splits; ++k) s += *reinterpret_cast<const f32x4*>(p + (int64_t)k * (Tl::BM * Tl::BN));
  store_y<Out>(Y, ldy, t, c, N, s);
}

// ---------------------------------------------------------------------------
// The same for up to 16 TF tokens: bound by reading the weights once.  A
// workgroup takes 16 RF channels, its wavefronts units of 16 blocks (512
// columns, 256 bytes of a row) in turn; lane l holds block 4 s + l / 16 of a
// unit for instruction s, and the 16 scale codes of the unit.  With kFused
// the activations are quantised here, a block a lane, in registers: one
// launch less, and each workgroup reads X itself (16-byte aligned rows).
// T = 1, 11008 x 4096: 9.6 us for 24 MB; the loads in flight, all issued at
// once, take about half of it, starting, summing and ending the rest.  The
// fused form's registers allow two workgroups a CU, 512 places for 688
// workgroups: a second round for the last 176.  T = 13, 4096 x 11008: 8.3 us
// for one workgroup a CU, whose wavefronts take two or three units one after
// another, loads and products of a unit in turn.
// ---------------------------------------------------------------------------
struct NoTokens {
  __device__ __forceinline__ NoTokens(const Adapters&, int64_t, int64_t) {}
};
template <int RF, int TF, class In, class Out, bool kFused, class Ad>
__global__ __launch_bounds__(kThinThreads, 4) void mx4_thin_kernel(Operand W, Operand Xq, const typename In::T* __restrict__ X,
                                                                int d, int ldx_bytes, int kchunks,
                                                                typename Out::T* __restrict__ Y, int64_t ldy,
                                                                Adapters ad) {
  __shared__ __align__(16) char red[thin_lds_bytes<RF, TF>()];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16 * RF;
  const uint32_t row_bytes = (uint32_t)kchunks * 16u;
  const int64_t ra = W.rows - m0 < 16 * RF ? W.rows - m0 : 16 * RF;
  const uint32_t pw = (uint32_t)W.pitch, sw = (uint32_t)W.scale_pitch;
  const __amdgpu_buffer_rsrc_t bufw = buffer_of(W.p + m0 * W.pitch, (uint32_t)((ra - 1) * W.pitch) + row_bytes),
                               bsw = buffer_of(W.scale + m0 * W.scale_pitch, (uint32_t)(ra * W.scale_pitch)),
                               bufr = buffer_of(X, kFused ? (uint32_t)(Xq.rows - 1) * (uint32_t)ldx_bytes + (uint32_t)d * sizeof(typename In::T) : 0u),
                               bufx = buffer_of(Xq.p, kFused ? 0 : (uint32_t)((Xq.rows - 1) * Xq.pitch) + row_bytes),
                               bsx = buffer_of(Xq.scale, kFused ? 0 : (uint32_t)(Xq.rows * Xq.scale_pitch));
  const int units = (kchunks + 15) / 16;
  f32x4 acc[RF][TF] = {};
  std::conditional_t<Ad::kOn, TokenAdapters<TF>, NoTokens> own(ad, l16, Xq.rows);
  for (int u = wave; u < units; u += kThinWaves) {
    i32x4 w[4][RF], sc[RF], x[4][TF], sx[TF];
    // Loads return in order: the activations first, so that they are quantised
    // while the weights are on their way.
    RawBlock<In> raw[kFused ? 4 : 1];
    if constexpr (kFused) {
      static_assert(TF == 1, "one token a lane");
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = 32 * (16 * u + 4 * s + g) + 8 * k;                  // d is a multiple of 8
          raw[s].r[k] = load16(bufr, j < d ? (uint32_t)(l16 * ldx_bytes) + 2u * j : kPastEnd, 0);
        }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t off = 16u * (4 * s + g);
        const bool in = 16 * u + 4 * s + g < kchunks;
#pragma unroll
        for (int j = 0; j < TF; ++j)
          x[s][j] = load16(bufx, in ? (uint32_t)(16 * j + l16) * (uint32_t)Xq.pitch + off : kPastEnd, (uint32_t)u * 256u);
      }
#pragma unroll
      for (int j = 0; j < TF; ++j) sx[j] = load16(bsx, (uint32_t)(16 * j + l16) * (uint32_t)Xq.scale_pitch, (uint32_t)u * 16u);
    }
#pragma unroll
    for (int i = 0; i < RF; ++i) sc[i] = load16(bsw, (uint32_t)(16 * i + l16) * sw, (uint32_t)u * 16u);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t off = 16u * (4 * s + g);
      const bool in = 16 * u + 4 * s + g < kchunks;
#pragma unroll
      for (int i = 0; i < RF; ++i) w[s][i] = load16(bufw, in ? (uint32_t)(16 * i + l16) * pw + off : kPastEnd, (uint32_t)u * 256u);
    }
    if constexpr (kFused) {
      __builtin_amdgcn_sched_barrier(0);
      sx[0] = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t code = scale_code(raw[s].max_bits());
        x[s][0] = raw[s].encode(code);
        sx[0][s] = (int)(code << (8 * g));
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int j = 0; j < TF; ++j)
          acc[i][j] = OpMx4::mma(w[s][i], x[s][j], acc[i][j], 0, (int)((uint32_t)sc[i][s] >> (8 * g)),
                                 (int)((uint32_t)sx[j][s] >> (8 * g)));
  }
  // the wavefronts take the tokens' adapters in turn, and their sums are added anyway
  if constexpr (Ad::kOn) add_adapters<Ad, kFused ? 1 : 4>(acc, ad, own, m0 + l16, l16, Xq.rows, W.rows, wave, kThinWaves);
  thin_sum(acc, red);
  if (wave) return;
#pragma unroll
  for (int j = 0; j < TF; ++j)
    if (16 * j + l16 < Xq.rows)
#pragma unroll
      for (int i = 0; i < RF; ++i)
        if (m0 + 16 * i + 4 * g < W.rows) store_y<Out>(Y, ldy, 16 * j + l16, m0 + 16 * i + 4 * g, W.rows, acc[i][j]);
}

// ===========================================================================
// launchers
// ===========================================================================
static void row_grid(int64_t N, int per_row, dim3* grid, dim3* block) {
  const int bx = std::min(kBlockThreads, (per_row + 63) / 64 * 64), by = kBlockThreads / bx;
  *block = dim3((unsigned)bx, (unsigned)by);
  *grid = dim3((unsigned)((per_row + bx - 1) / bx), (unsigned)std::min<int64_t>((N + by - 1) / by, 65535));
}

template <class In, class Val>
static int quantize_as(const void* W, int64_t N, int d, int64_t ldw, uint8_t* codes, uint8_t* scales, void* values,
                       int64_t ldv, hipStream_t st) {
  dim3 grid, block;
  const int nb = (int)mx4_blocks(d);
  row_grid(N, 4 * nb, &grid, &block);
  // fp32 rows of some length go two groups a lane, where there are enough lanes all the same: 4095 x 11007 with
  // fp32 values 75 us against 84 us (bf16 is slower that way: 39.3 against 38.0 us at 4096 x 11008)
  constexpr int kMost = sizeof(typename In::T) == 4 ? 2 : 1;
  const bool many = kMost > 1 && grid.x > 1 && (int64_t)grid.x * std::min<int64_t>(tiles_of(N, block.y), 65535) >= 32 * kCus;
  if (many) grid.x = (unsigned)tiles_of(grid.x, kMost);
  auto kernel = many ? mx4_quantize_kernel<In, Val, kMost> : mx4_quantize_kernel<In, Val, 1>;
  hipLaunchKernelGGL(kernel, grid, block, 0, st, (const typename In::T*)W, N, d, ldw, codes, scales, nb,
                     (int)mx4_scale_bytes(d), (typename Val::T*)values, ldv);
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
                     (typename Out::T*)W, ldo);
  return check_launch("mx4_dequantize_kernel");
}
int launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t N, int d, void* W, int32_t odt,
                          int64_t ldo, hipStream_t st) {
  if (odt == QAMW_F32) return dequantize_to<MemF32>(codes, scales, N, d, W, ldo, st);
  if (odt == QAMW_F16) return dequantize_to<MemF16>(codes, scales, N, d, W, ldo, st);
  return dequantize_to<MemBf16>(codes, scales, N, d, W, ldo, st);
}

// Sizes and places of the product's workspace: the quantised activations and
// the results of split tiles.
struct Mx4Plan {
  TailPlan tiles;
  size_t scales, part, bytes;
};
// Whether the weights are read in thin tiles: up to 16 tokens, and up to 32
// where 64 x 64 tiles would leave half the CUs idle (T = 32: 4096 x 4096 10.2
// us thin, 12.6 us tiled; 11008 x 4096 16.2 us and 13.4 us).
static bool thin_pays(int64_t T, int64_t N) { return T <= 16 || (T <= 32 && 2 * tiles_of(N, 64) <= kCus); }
static Mx4Plan mx4_plan(int64_t T, int64_t N, int64_t d) {
  Mx4Plan p;
  p.tiles = {0, 0, 1};
  p.scales = round_up((size_t)T * mx4_blocks(d) * 16, 256);
  p.part = p.scales + round_up((size_t)T * mx4_scale_bytes(d), 256);
  p.bytes = p.part;
  if (!thin_pays(T, N)) {
    p.tiles = tail_plan(kProductMx4, N, T, tiles_of(mx4_blocks(d), kStepChunks));
    const int64_t tile = kShapeTile[p.tiles.shape], tail = shape_tiles(p.tiles.shape, N, T) - p.tiles.whole;
    p.bytes += (size_t)(tail * p.tiles.splits * tile * tile) * sizeof(float);
  }
  return p;
}
bool mx4_grid_fits(int64_t T, int64_t N, int64_t d) {
  // below these no shape comes near the limit: less than 2^22 tiles
  if (T < (int64_t(1) << 26) && N < (int64_t(1) << 26) && T * N < (int64_t(1) << 31)) return true;
  if (thin_pays(T, N)) return grid_holds(tiles_of(N, 16), kThinThreads);
  const TailPlan p = mx4_plan(T, N, d).tiles;
  const int64_t n = shape_tiles(p.shape, N, T);
  return grid_holds(p.whole + (n - p.whole) * p.splits, shape_threads(p.shape));
}
size_t mx4_matmul_workspace_bytes(int64_t T, int64_t N, int64_t d) { return mx4_plan(T, N, d).bytes; }
// Whether the adapters' part of Y is written as a matrix first, which the
// product's sums start from.  A tile's workgroup multiplies the adapters of its
// tokens one after another: nothing where the tokens of a prompt share one,
// but too much in a batch whose tokens have one each (48 of rank 16 beside 4096
// x 4096: 31 us in the product's 64 workgroups).  Past 256 tokens the matrix in
// fp32 costs more than that where tokens share adapters (4095 x 13824: 226 MB
// written and read; 256 and 257 tokens of one adapter, 4096 x 4096: 32 us and 26
// us), and much less where they do not (of 64 adapters in turn: 48 us and 361
// us), which the host does not know.  Tiles copy B by 16-byte chunks and hold U
// in bf16: fp32, and ranks of no whole chunks unless launch_adapter_shrink fills
// them up, go by the matrix.
bool adapters_in_delta(int64_t T, int64_t N, int32_t dt, int64_t rank) {
  return !thin_pays(T, N) && (T <= 256 || dt == QAMW_F32 || rank % 8 != 0);
}

template <class Tl, class Out, class Ad>
static int matmul_tiled(const TailPlan& p, const Operand& W, const Operand& X, int kchunks, void* Y, int64_t ldy, float* part,
                        const Adapters& ad, hipStream_t st) {
  typedef typename Out::T E;
  const int tm = (int)tiles_of(W.rows, Tl::BM), tn = (int)tiles_of(X.rows, Tl::BN), whole = (int)p.whole, tail = tm * tn - whole;
  auto kernel = mx4_matmul_kernel<Tl, Out, Ad>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(whole + tail * p.splits)), dim3(Tl::kThreads), Tl::kLdsBytes, st, W, X, kchunks,
                     tm, tn, whole, p.splits, (E*)Y, ldy, part, ad);
  const int rc = check_launch("mx4_matmul_kernel");
  if (rc || !tail) return rc;
  auto sum = mx4_sum_tail_kernel<Tl, Out>;
  hipLaunchKernelGGL(sum, dim3((unsigned)(Tl::BM * Tl::BN / 1024), (unsigned)tail), dim3(256), 0, st, part, whole, p.splits, tm,
                     tn, X.rows, W.rows, (E*)Y, ldy);
  return check_launch("mx4_sum_tail_kernel");
}
template <class Out, class Ad>
static int matmul_to(const TailPlan& p, const Operand& W, const Operand& X, int kchunks, void* Y, int64_t ldy, float* part,
                     const Adapters& ad, hipStream_t st) {
  return with_shape<OpMx4>(
      p.shape, [&](auto tile) { return matmul_tiled<decltype(tile), Out, Ad>(p, W, X, kchunks, Y, ldy, part, ad, st); });
}

// A workgroup of the thin product takes 32 channels where that still gives
// every CU one, else 16 (T = 13: 4096 x 11008 13.5 us with 16, 16.3 us with
// 32; T = 16: 11008 x 4096 13.6 us with 32).  The fused form takes 16: its
// registers allow two workgroups a CU only then (T = 1, 11008 x 4096: 10.9 us
// against 12.1 us).
template <int RF, int TF, class In, class Out, bool kFused, class Ad>
static int thin_rows(const Operand& W, const Operand& Xq, const void* X, int d, int64_t ldx, int kchunks, void* Y, int64_t ldy,
                     const Adapters& ad, hipStream_t st) {
  hipLaunchKernelGGL((mx4_thin_kernel<RF, TF, In, Out, kFused, Ad>), dim3((unsigned)tiles_of(W.rows, 16 * RF)), dim3(kThinThreads),
                     0, st, W, Xq, (const typename In::T*)X, d, (int)(ldx * sizeof(typename In::T)), kchunks,
                     (typename Out::T*)Y, ldy, ad);
  return check_launch("mx4_thin_kernel");
}
template <int TF, class In, class Out, bool kFused, class Ad>
static int matmul_thin(const Operand& W, const Operand& Xq, const void* X, int d, int64_t ldx, int kchunks, void* Y, int64_t ldy,
                       const Adapters& ad, hipStream_t st) {
  if constexpr (!kFused && TF == 1)
    if (tiles_of(W.rows, 32) >= kCus) return thin_rows<2, TF, In, Out, kFused, Ad>(W, Xq, X, d, ldx, kchunks, Y, ldy, ad, st);
  return thin_rows<1, TF, In, Out, kFused, Ad>(W, Xq, X, d, ldx, kchunks, Y, ldy, ad, st);
}
template <class Out, class Ad>
static int matmul_quantised(const Mx4Plan& p, const Operand& W, const Operand& X, int d, int kchunks, void* Y, int64_t ldy,
                            float* part, const Adapters& ad, hipStream_t st) {
  if (X.rows <= 16) return matmul_thin<1, MemBf16, Out, false, Ad>(W, X, nullptr, d, 0, kchunks, Y, ldy, ad, st);
  if (thin_pays(X.rows, W.rows)) return matmul_thin<2, MemBf16, Out, false, Ad>(W, X, nullptr, d, 0, kchunks, Y, ldy, ad, st);
  auto by_matrix = [&](int32_t dt) {
    const int rc = launch_adapter_expand(dt, X.rows, W.rows, ad, st);
    return rc ? rc : matmul_to<Out, AdapterDelta>(p.tiles, W, X, kchunks, Y, ldy, part, ad, st);
  };
  if constexpr (std::is_same<Ad, AdaptersF32>::value) {
    return by_matrix(QAMW_F32);                    // adapters_in_delta is true of fp32 here
  } else {
    if constexpr (Ad::kOn)
      if (adapters_in_delta(X.rows, W.rows, QAMW_BF16, ad.rank)) return by_matrix(QAMW_BF16);
    return matmul_to<Out, Ad>(p.tiles, W, X, kchunks, Y, ldy, part, ad, st);
  }
}

// Up to this many tokens of 16 bits the thin product quantises X itself: each
// of its workgroups then reads no more of X than of the weights (4096 x 4096,
// T = 1: 5.4 us against 7.0 us with a launch of its own for X).
constexpr int64_t kFusedTokens = 4;

template <class Out>
static int matmul_out(const void* X, int32_t xdt, int64_t T, int d, int64_t ldx, const uint8_t* wcodes, const uint8_t* wscales,
                      int64_t N, void* Y, int64_t ldy, void* ws, const Adapters* adapters, hipStream_t st) {
  const int nb = (int)mx4_blocks(d), es = elem_size(xdt);
  const Mx4Plan p = mx4_plan(T, N, d);
  uint8_t *xcodes = (uint8_t*)ws, *xscales = xcodes + p.scales;
  float* part = (float*)(xcodes + p.part);
  const Operand w = {(const char*)wcodes, (int64_t)nb * 16, N, wscales, mx4_scale_bytes(d)};
  const Operand x = {(const char*)xcodes, (int64_t)nb * 16, T, xscales, mx4_scale_bytes(d)};
  const Adapters ad = adapters ? *adapters : Adapters{};
  typedef std::conditional_t<sizeof(typename Out::T) == 4, AdaptersBf16x3, AdaptersBf16> AdBf16;
  // the fused form reads X by 16-byte loads with 32-bit offsets
  if (T <= kFusedTokens && es == 2 && d % 8 == 0 && aligned16(X) && ldx % 8 == 0 && ldx <= kMaxRowBytes / es) {
    if (xdt == QAMW_F16) return matmul_thin<1, MemF16, Out, true, NoAdapters>(w, x, X, d, ldx, nb, Y, ldy, ad, st);
    if (adapters) return matmul_thin<1, MemBf16, Out, true, AdBf16>(w, x, X, d, ldx, nb, Y, ldy, ad, st);
    return matmul_thin<1, MemBf16, Out, true, NoAdapters>(w, x, X, d, ldx, nb, Y, ldy, ad, st);
  }
  const int rc = launch_mx4_quantize(X, xdt, T, d, ldx, xcodes, xscales, nullptr, QAMW_BF16, 0, st);
  if (rc) return rc;
  if (!adapters) return matmul_quantised<Out, NoAdapters>(p, w, x, d, nb, Y, ldy, part, ad, st);
  if (xdt == QAMW_F32) return matmul_quantised<Out, AdaptersF32>(p, w, x, d, nb, Y, ldy, part, ad, st);
  return matmul_quantised<Out, AdBf16>(p, w, x, d, nb, Y, ldy, part, ad, st);
}
int launch_mx4_matmul(const void* X, int32_t xdt, int64_t T, int d, int64_t ldx, const uint8_t* wcodes,
                      const uint8_t* wscales, int64_t N, void* Y, int32_t ydt, int64_t ldy, void* ws,
                      const Adapters* adapters, hipStream_t st) {
  return ydt == QAMW_F32 ? matmul_out<MemF32>(X, xdt, T, d, ldx, wcodes, wscales, N, Y, ldy, ws, adapters, st)
                         : matmul_out<MemBf16>(X, xdt, T, d, ldx, wcodes, wscales, N, Y, ldy, ws, adapters, st);
}

}  // namespace qamw
