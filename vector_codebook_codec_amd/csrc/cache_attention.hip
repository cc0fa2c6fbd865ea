// Attention over the cache in microscaled 4-bit floating point (cache.hip has
// its layout): for a query row of a sequence with n queries and `length`
// cached tokens, the i-th query at place length - n + i,
//     z_t = scale <q, k_t>,  out = sum_t softmax(z)_t v_t,  lse = log sum_t exp z_t
// over the tokens that the masks leave: t < length, t <= place (causal),
// t > place - window.  A row that is left none gives 0 and -infinity.
#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "mx4_device.h"
#include "qamw.h"
#include "qamw_device.h"
#include "qamw_internal.h"

namespace qamw {

constexpr int kAttnWaves = 4, kAttnThreads = kAttnWaves * kWave;
constexpr int kWaveTokens = 32, kTileTokens = kAttnWaves * kWaveTokens;
constexpr int kMaxSplits = 64;                     // a wavefront joins them, one a lane
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// A sequence's queries and cached tokens, whatever the arrays hold: queries
// stay inside [0, T), tokens inside the page table.
struct Sequence {
  int64_t first;                                   // its first query
  int n, length;
};
__device__ __forceinline__ Sequence sequence_of(const AttentionArgs& a, int b) {
  Sequence s;
  if (a.starts) {
    const int64_t s0 = a.starts[b], s1 = a.starts[b + 1];
    s.first = s0 < 0 ? 0 : s0 > a.T ? a.T : s0;
    s.n = (int)((s1 > a.T ? a.T : s1) - s.first);
  } else {
    s.first = b;
    s.n = b < a.T ? 1 : 0;
  }
  s.n = s.n > 0 ? s.n : 0;
  const int64_t most = (int64_t)a.cols << a.c.page_shift, len = a.lengths[b];
  s.length = (int)(len < 0 ? 0 : len > most ? most : len);
  return s;
}
// the tokens [lo, hi) that query i of a sequence attends to (hi below lo: none)
__device__ __forceinline__ int span_end(const AttentionArgs& a, const Sequence& s, int i) {
  const int end = s.length - s.n + i + 1;
  return a.causal && end < s.length ? end : s.length;
}
__device__ __forceinline__ int span_begin(const AttentionArgs& a, const Sequence& s, int i) {
  const int begin = s.length - s.n + i + 1 - a.window;
  return a.window && begin > 0 ? begin : 0;
}
// The token tiles of query rows [r0, r1) and into how many shares they go.
struct TileRange {
  int first, count, shares;
};
__device__ __forceinline__ TileRange tile_range(const AttentionArgs& a, const Sequence& s, int r0, int r1, int splits) {
  const int lo = span_begin(a, s, r0 / a.group), hi = span_end(a, s, (r1 - 1) / a.group);
  TileRange t;
  t.first = lo / kTileTokens;
  t.count = hi > lo ? (hi + kTileTokens - 1) / kTileTokens - t.first : 0;
  t.shares = t.count < splits ? (t.count > 1 ? t.count : 1) : splits;
  return t;
}

__device__ __forceinline__ void load8_as(int32_t dt, const void* row, int j, int d, float (&x)[8]) {
  if (dt == QAMW_F32) load8<MemF32>((const float*)row, j, d, x);
  else if (dt == QAMW_F16) load8<MemF16>((const uint16_t*)row, j, d, x);
  else load8<MemBf16>((const uint16_t*)row, j, d, x);
}
__device__ __forceinline__ void store8_as(int32_t dt, void* row, int j, int d, const float (&x)[8]) {
  if (dt == QAMW_F32) store8<MemF32>((float*)row, j, d, x);
  else if (dt == QAMW_F16) store8<MemF16>((uint16_t*)row, j, d, x);
  else store8<MemBf16>((uint16_t*)row, j, d, x);
}
__device__ __forceinline__ void* row_at(const void* p, int32_t dt, int64_t element) {
  return (char*)const_cast<void*>(p) + element * (dt == QAMW_F32 ? 4 : 2);
}

// the 8 four-bit elements of w times the scale, as bf16 (exact)
__device__ __forceinline__ void decode_bf16(uint32_t w, float s, uint32_t (&o)[4]) {
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
}
// x as a sum of kTerms bf16 numbers: 8, 16 or 24 bits of it
template <int kTerms>
__device__ __forceinline__ void split_bf16x2(float x0, float x1, uint32_t (&o)[kTerms]) {
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    o[t] = pack_bf16x2(x0, x1);
    if (t + 1 < kTerms) x0 -= __uint_as_float(o[t] << 16), x1 -= __uint_as_float(o[t] & 0xffff0000u);
  }
}
__device__ __forceinline__ f32x4 mfma_bf16(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// floats of a share's partial result: sums, then the reference exponent and the sum of weights of each row
template <int DB, int RT> constexpr int part_floats() { return 16 * RT * (32 * DB + 2); }

// ---------------------------------------------------------------------------
// A workgroup takes 16 RT query rows (query by head of the group) of one
// sequence and key head and one share of their tokens, 128 at a time; each of
// its 4 wavefronts takes 32 of these tokens, and their results are joined at
// the end.  DB: heads of up to 32 DB elements.  Everything goes from global
// memory straight into the registers that the matrix instructions read:
//   * S^T = K Q^T: lane l holds the token l % 16 and 8 DB consecutive elements
//     of it, decoded to bf16 (4-bit values by a power of two are exact there).
//     A lane then has scores of one query row, l % 16, and of 4 tokens, 4 (l /
//     16) + r: a row's running maximum and sum are one register.
//   * O^T = V^T P^T: the scores of two groups of 16 tokens are in place as the
//     operand P.  Lane l decodes elements 2 DB (l % 16) + (0 .. 2 DB - 1) of
//     the same 8 tokens, pairs of tokens are put together by byte permutes,
//     and the m-th instruction multiplies the m-th element of every lane.
// The reference of the exponentials follows the maximum only when a score
// exceeds it by 2^8 (they are then up to 256, far from any limit): nearly all
// tiles go without an exchange between lanes and without a pass over the sums.
//
// kTerms: q and the weights p are sums of that many bf16 numbers: 1 for bf16
// in and out (p rounded by at most 2^-8 of itself, each weight on its own; as
// much as the output's own rounding), 2 where fp16 and 3 where fp32 takes part
// (p to 2^-16 and 2^-24).  Sums are fp32 throughout.
// ---------------------------------------------------------------------------
template <int DB, int RT, int kTerms>
__global__ __launch_bounds__(kAttnThreads) void cache_attention_kernel(AttentionArgs a, int row_tiles, int splits,
                                                                       float* __restrict__ part) {
  constexpr int MT = 2 * DB;                       // matrix instructions along the head
  constexpr int VW = DB == 8 ? 2 : 1;              // words of a token's elements in one lane
  constexpr int LD = 32 * DB + 4;                  // LDS row, off the banks' period
  __shared__ __align__(16) float joined[kAttnWaves * 16 * LD];
  __shared__ float stats[2][kAttnWaves][16];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Workgroup -> (sequence and key head, row tile, share).  Where the pairs
  // divide among the 8 XCDs, all work of a pair goes to one: its keys and
  // values then pass through one L2.  The last rows, which see most tokens, first.
  const int pairs = a.sequences * a.c.heads, per = row_tiles * splits, id = blockIdx.x;
  int pair, inner;
  if (pairs % 8 == 0) pair = id / 8 / per * 8 + id % 8, inner = id / 8 % per;
  else pair = id / per, inner = id % per;
  const int b = pair / a.c.heads, h = pair - b * a.c.heads;
  const int tile = row_tiles - 1 - inner / splits, share = inner % splits;
  const Sequence seq = sequence_of(a, b);
  const int rows = min((int64_t)seq.n * a.group, (int64_t)INT32_MAX), r0 = tile * 16 * RT, r1 = min(rows, r0 + 16 * RT);
  if (r0 >= rows) return;
  const TileRange range = tile_range(a, seq, r0, r1, splits);
  if (share >= range.shares) return;
  const int k0 = range.first + (int)((int64_t)range.count * share / range.shares),
            k1 = range.first + (int)((int64_t)range.count * (share + 1) / range.shares);
  // tokens of any row, and of every row
  const int lo_any = span_begin(a, seq, r0 / a.group), hi_any = span_end(a, seq, (r1 - 1) / a.group);
  const int lo_all = span_begin(a, seq, (r1 - 1) / a.group), hi_all = span_end(a, seq, r0 / a.group);

  // ---- queries, and the span of this lane's row of each tile of 16
  i32x4 q[RT][DB][kTerms];
  int row_lo[RT], row_hi[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int row = r0 + 16 * j + l16, i = min(row, r1 - 1) / a.group, head = h * a.group + min(row, r1 - 1) % a.group;
    row_lo[j] = span_begin(a, seq, i), row_hi[j] = span_end(a, seq, i);
    const void* p = row_at(a.Q, a.qdt, (seq.first + i) * a.q_token + head * a.q_head);
#pragma unroll
    for (int w = 0; w < DB; ++w) {
      float x[8];
      load8_as(a.qdt, p, 8 * (g * DB + w), a.c.d, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t t[kTerms];
        split_bf16x2<kTerms>(x[2 * e], x[2 * e + 1], t);
#pragma unroll
        for (int k = 0; k < kTerms; ++k) q[j][w][k][e] = (int)t[k];
      }
    }
  }

  f32x4 o[RT][MT] = {};
  float m[RT], l[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) m[j] = -FLT_MAX, l[j] = 0.0f;

  // ---- loads of this wavefront's 32 tokens of tile k, two groups of 16; a
  // page outside the cache, a group outside every row's span and elements past
  // the head read as 0
  struct Raw {
    uint32_t k[2][DB], ks[2], v[2][4][VW], vs[2][DB];
    bool page_ok[2];
  };
  typedef const __attribute__((address_space(4))) int32_t* ConstantInts;
  const ConstantInts table = (ConstantInts)(uintptr_t)(a.table + b * a.table_pitch);
  const int rb = 16 * a.c.nb, shift = a.c.page_shift, in_page = (1 << shift) - 1;
  const uint32_t page_codes = (uint32_t)rb << shift, page_scales = (uint32_t)a.c.sb << shift;
  const int64_t v_codes = a.c.pages * a.c.heads * (int64_t)page_codes, v_scales = a.c.pages * a.c.heads * (int64_t)page_scales;
  auto pages_of = [&](int k, int (&page)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = k * kTileTokens + wave * kWaveTokens + 16 * i;
      page[i] = k < k1 && t < hi_any && t + 16 > lo_any ? table[t >> shift] : -1;
    }
  };
  const uint32_t k_at = (uint32_t)(l16 * rb + g * (4 * DB)), v_at = (uint32_t)(4 * g * rb + l16 * DB);
  const uint32_t ks_at = (uint32_t)(l16 * a.c.sb + (DB == 2 ? g >> 1 : DB == 4 ? g : 2 * g));
  auto load = [&](int k, const int (&page)[2], Raw& r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool ok = page[i] >= 0 && page[i] < a.c.pages;
      r.page_ok[i] = ok;
      const int64_t block = (int64_t)(ok ? page[i] : 0) * a.c.heads + h;
      const uint8_t *pc = a.codes + block * page_codes, *ps = a.scales + block * page_scales;
      const __amdgpu_buffer_rsrc_t bk = buffer_of(pc, ok ? page_codes : 0), bks = buffer_of(ps, ok ? page_scales : 0),
                                   bv = buffer_of(pc + v_codes, ok ? page_codes : 0),
                                   bvs = buffer_of(ps + v_scales, ok ? page_scales : 0);
      // scalar offsets stay inside the buffer: the range check subtracts them from its size
      const int at = ok ? k * kTileTokens + wave * kWaveTokens + 16 * i & in_page : 0;
      const int sc = at * rb, ss = at * a.c.sb;
#pragma unroll
      for (int w = 0; w < DB; w += 4) {            // 16 bytes (8 with DB = 2), a whole or no part of a block
        const int off = (int)(g * 4 * DB + 4 * w < rb ? k_at + 4 * w : kPastEnd);
        if constexpr (DB == 2) {
          const auto x = __builtin_amdgcn_raw_buffer_load_b64(bk, off, sc, 0);
          r.k[i][0] = (uint32_t)x[0], r.k[i][1] = (uint32_t)x[1];
        } else {
          const auto x = __builtin_amdgcn_raw_buffer_load_b128(bk, off, sc, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) r.k[i][w + e] = (uint32_t)x[e];
        }
      }
      if constexpr (DB == 8) r.ks[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(bks, (int)ks_at, ss, 0);
      else r.ks[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(bks, (int)ks_at, ss, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int off = (int)(l16 * DB < rb ? v_at + e * rb : kPastEnd);
        if constexpr (DB == 2) {
          r.v[i][e][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(bv, off, sc, 0);
        } else if constexpr (DB == 4) {
          r.v[i][e][0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(bv, off, sc, 0);
        } else {
          const auto x = __builtin_amdgcn_raw_buffer_load_b64(bv, off, sc, 0);
          r.v[i][e][0] = (uint32_t)x[0], r.v[i][e][VW - 1] = (uint32_t)x[1];
        }
      }
      // the scale codes of 4 tokens in a row
      if constexpr (DB == 2) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b64(bvs, 8 * g, ss, 0);
        r.vs[i][0] = (uint32_t)x[0], r.vs[i][1] = (uint32_t)x[1];
      } else {
#pragma unroll
        for (int w = 0; w < DB; w += 4) {
          const auto x = __builtin_amdgcn_raw_buffer_load_b128(bvs, 4 * DB * g + 4 * w, ss, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) r.vs[i][w + e] = (uint32_t)x[e];
        }
      }
    }
  };

  const float c = a.scale * kLog2e;
  auto compute = [&](int k, const Raw& r) __attribute__((always_inline)) {
    const int t0 = k * kTileTokens + wave * kWaveTokens;
    // ---- scores
    f32x4 s[RT][2] = {};
#pragma unroll
    for (int w = 0; w < DB; ++w) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t kd[4];
        decode_bf16(r.k[i][w], __uint_as_float((DB == 8 && w < 4 ? r.ks[i] & 255u : DB == 8 ? r.ks[i] >> 8 : r.ks[i]) << 23), kd);
        const i32x4 kf = {(int)kd[0], (int)kd[1], (int)kd[2], (int)kd[3]};
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int t = 0; t < kTerms; ++t) s[j][i] = mfma_bf16(kf, q[j][w][t], s[j][i]);
      }
    }
    // ---- masks: whether every row sees all 32 tokens, and if not, which
    const bool whole = t0 >= lo_all && t0 + kWaveTokens <= hi_all && r.page_ok[0] && r.page_ok[1];
    auto sees = [&](int j, int i, int e) __attribute__((always_inline)) {
      const int t = t0 + 16 * i + 4 * g + e;
      return t >= row_lo[j] && t < row_hi[j] && r.page_ok[i];
    };
    if (!whole) {
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(j, i, e)) s[j][i][e] = -INFINITY;
    }
    // ---- the reference of the exponentials
    float top[RT];
    bool above = false;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const float x = fmaxf(fmaxf(s[j][0][0], s[j][0][1]), fmaxf(s[j][0][2], s[j][0][3])),
                  y = fmaxf(fmaxf(s[j][1][0], s[j][1][1]), fmaxf(s[j][1][2], s[j][1][3]));
      top[j] = fmaxf(x, y) * c;
      above |= top[j] > m[j] + 8.0f;
    }
    if (__ballot(above)) {
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        float x = fmaxf(top[j], __shfl_xor(top[j], 16));
        x = fmaxf(m[j], fmaxf(x, __shfl_xor(x, 32)));
        const float f = __builtin_amdgcn_exp2f(m[j] - x);
        m[j] = x;
        l[j] *= f;
#pragma unroll
        for (int t = 0; t < MT; ++t) o[j][t] *= f;
      }
    }
    // ---- weights
    i32x4 p[RT][kTerms];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i][e], c, -m[j])),
                      p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i][e + 1], c, -m[j]));
          l[j] += p0 + p1;
          uint32_t t[kTerms];
          split_bf16x2<kTerms>(p0, p1, t);
#pragma unroll
          for (int n = 0; n < kTerms; ++n) p[j][n][2 * i + e / 2] = (int)t[n];
        }
    }
    // ---- values: scale codes of this lane's block for its 8 tokens
    uint32_t vc[8], vw[8][VW];
    const int block = l16 * DB / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (DB == 2) vc[4 * i + e] = r.vs[i][e / 2] >> (16 * (e & 1) + 8 * block) & 255u;
        if constexpr (DB == 4) vc[4 * i + e] = r.vs[i][e] >> (8 * block) & 255u;
        if constexpr (DB == 8) vc[4 * i + e] = (block < 4 ? r.vs[i][2 * e] : r.vs[i][2 * e + 1]) >> (8 * (block & 3)) & 255u;
#pragma unroll
        for (int n = 0; n < VW; ++n) vw[4 * i + e][n] = r.v[i][e][n];
      }
    // tokens that no row sees may hold anything
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + 16 * i + 4 * g + e;
          if (t < lo_any || t >= hi_any) {
            vc[4 * i + e] = 0;
#pragma unroll
            for (int n = 0; n < VW; ++n) vw[4 * i + e][n] = 0;
          }
        }
    }
    // Blocks that are NaN must reach the rows that see their token and no
    // others, whose weight of it is 0: they are taken as 0, and the elements of
    // a row become NaN where the product of "sees the token" and "is NaN" counts any.
    uint32_t most = vc[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) most = max(most, vc[e]);
    if (__ballot(most == 255u)) {
      i32x4 bad = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (vc[e] == 255u) {
          bad[e / 2] |= 0x3f80 << (16 * (e & 1));
          vc[e] = 0;
#pragma unroll
          for (int n = 0; n < VW; ++n) vw[e][n] = 0;
        }
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        i32x4 seen = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (sees(j, e / 4, e & 3)) seen[e / 2] |= 0x3f80 << (16 * (e & 1));
        const f32x4 count = mfma_bf16(bad, seen, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (count[e] > 0.0f)
#pragma unroll
            for (int t = 0; t < MT; ++t) o[j][t][e] = NAN;
      }
    }
    // ---- O^T += V^T P^T, two elements of the head at a time from one byte of every token
#pragma unroll
    for (int n = 0; n < VW; ++n) {
      uint32_t d[8][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) decode_bf16(vw[e][n], __uint_as_float(vc[e] << 23), d[e]);
#pragma unroll
      for (int x = 0; x < (DB == 2 ? 2 : 4); ++x) {
        i32x4 even, odd;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          even[e] = (int)__builtin_amdgcn_perm(d[2 * e + 1][x], d[2 * e][x], 0x05040100);
          odd[e] = (int)__builtin_amdgcn_perm(d[2 * e + 1][x], d[2 * e][x], 0x07060302);
        }
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int t = 0; t < kTerms; ++t) {
            o[j][8 * n + 2 * x] = mfma_bf16(even, p[j][t], o[j][8 * n + 2 * x]);
            o[j][8 * n + 2 * x + 1] = mfma_bf16(odd, p[j][t], o[j][8 * n + 2 * x + 1]);
          }
      }
    }
  };

  // ---- the tiles, the next one's loads in flight while one is computed, the one after's pages too
  if (k0 < k1) {
    Raw raw[2];
    int page[2];
    pages_of(k0, page);
    load(k0, page, raw[0]);
    pages_of(k0 + 1, page);
    for (int k = k0; k < k1; k += 2) {
      load(k + 1, page, raw[1]);
      pages_of(k + 2, page);
      compute(k, raw[0]);
      if (k + 1 >= k1) break;
      load(k + 2, page, raw[0]);
      pages_of(k + 3, page);
      compute(k + 1, raw[1]);
    }
  }

  // ---- join the wavefronts, 16 rows at a time
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    l[j] += __shfl_xor(l[j], 16);
    l[j] += __shfl_xor(l[j], 32);
    if (j) __syncthreads();                        // the last 16 rows have been read
    if (g == 0) stats[0][wave][l16] = m[j];
    __syncthreads();
    float top = stats[0][0][l16];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, stats[0][w][l16]);
    const float f = __builtin_amdgcn_exp2f(m[j] - top);
    if (g == 0) stats[1][wave][l16] = l[j] * f;
    float* to = joined + (wave * 16 + l16) * LD + MT * 4 * g;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int t = 0; t < MT; t += 4)
        *reinterpret_cast<f32x4*>(to + MT * e + t) = f32x4{o[j][t][e], o[j][t + 1][e], o[j][t + 2][e], o[j][t + 3][e]} * f;
    __syncthreads();
    const int sub = threadIdx.x >> 4, at = (threadIdx.x & 15) * MT, row = r0 + 16 * j + sub;
    if (row >= r1) continue;
    float x[MT], sum = 0.0f, ref = stats[0][0][sub];
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      sum += stats[1][w][sub];
      ref = fmaxf(ref, stats[0][w][sub]);
#pragma unroll
      for (int t = 0; t < MT; t += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(joined + (w * 16 + sub) * LD + at + t);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t + e] += v[e];
      }
    }
    if (range.shares > 1) {
      float* to_part = part + (((int64_t)pair * row_tiles + tile) * splits + share) * part_floats<DB, RT>();
#pragma unroll
      for (int t = 0; t < MT; t += 4)
        *reinterpret_cast<f32x4*>(to_part + (16 * j + sub) * 32 * DB + at + t) = f32x4{x[t], x[t + 1], x[t + 2], x[t + 3]};
      if ((threadIdx.x & 15) == 0) {
        to_part[16 * RT * 32 * DB + 16 * j + sub] = ref;
        to_part[16 * RT * (32 * DB + 1) + 16 * j + sub] = sum;
      }
      continue;
    }
    const int64_t query = seq.first + row / a.group;
    const int head = h * a.group + row % a.group;
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;         // NaN stays NaN
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] *= inv;
    void* to_out = row_at(a.out, a.odt, query * a.o_token + head * a.o_head);
    if constexpr (MT == 4) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (at + t < a.c.d) {
          if (a.odt == QAMW_F32) ((float*)to_out)[at + t] = x[t];
          else ((uint16_t*)to_out)[at + t] = a.odt == QAMW_F16 ? MemF16::put(x[t]) : MemBf16::put(x[t]);
        }
    } else {
#pragma unroll
      for (int t = 0; t < MT; t += 8) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[t + e];
        store8_as(a.odt, to_out, at + t, a.c.d, y);
      }
    }
    if (a.lse && (threadIdx.x & 15) == 0)
      a.lse[query * a.c.heads * a.group + head] = sum != 0.0f ? (ref + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
  }
}

// Rows whose tokens went into several shares: a wavefront a row.
template <int DB>
__global__ __launch_bounds__(kAttnThreads) void cache_attention_join_kernel(AttentionArgs a, int tile_rows, int row_tiles,
                                                                            int splits, const float* __restrict__ part) {
  const int lane = threadIdx.x & (kWave - 1), heads = a.c.heads * a.group;
  const int64_t id = (int64_t)blockIdx.x * kAttnWaves + (threadIdx.x >> 6), query = id / heads;
  const int head = (int)(id - query * heads), h = head / a.group;
  if (query >= a.T) return;
  int b = (int)query;
  if (a.starts) {                                  // the last sequence that starts at or before the query
    int lo = 0, hi = a.sequences;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (a.starts[mid] <= query) lo = mid + 1;
      else hi = mid;
    }
    b = lo - 1;
  }
  if (b < 0 || b >= a.sequences) return;
  const Sequence seq = sequence_of(a, b);
  if (query < seq.first || query >= seq.first + seq.n) return;
  const int64_t row = (query - seq.first) * a.group + (head - h * a.group);
  const int tile = (int)(row / tile_rows), r0 = tile * tile_rows;
  if (tile >= row_tiles) return;
  const int r1 = (int)min((int64_t)seq.n * a.group, (int64_t)r0 + tile_rows);
  const TileRange range = tile_range(a, seq, r0, r1, splits);
  if (range.shares <= 1) return;                   // written already
  const int64_t floats = (int64_t)tile_rows * (32 * DB + 2);
  const float* p = part + (((int64_t)b * a.c.heads + h) * row_tiles + tile) * splits * floats;
  const int at = (int)(row - r0);
  const float ref = lane < range.shares ? p[lane * floats + tile_rows * 32 * DB + at] : -FLT_MAX;
  float top = ref, sum = lane < range.shares ? p[lane * floats + tile_rows * (32 * DB + 1) + at] : 0.0f;
#pragma unroll
  for (int x = 1; x < kWave; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
  const float f = __builtin_amdgcn_exp2f(ref - top);
  sum *= f;
#pragma unroll
  for (int x = 1; x < kWave; x *= 2) sum += __shfl_xor(sum, x);
  constexpr int E = DB / 2;                        // elements of a lane
  float acc[E] = {};
  for (int s = 0; s < range.shares; ++s) {
    const float fs = __shfl(f, s);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += fs * p[s * floats + at * 32 * DB + E * lane + e];
  }
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  void* to = row_at(a.out, a.odt, query * a.o_token + head * a.o_head);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (E * lane + e < a.c.d) {
      const float x = acc[e] * inv;
      if (a.odt == QAMW_F32) ((float*)to)[E * lane + e] = x;
      else ((uint16_t*)to)[E * lane + e] = a.odt == QAMW_F16 ? MemF16::put(x) : MemBf16::put(x);
    }
  if (a.lse && lane == 0) a.lse[query * heads + head] = sum != 0.0f ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
}

// ===========================================================================
// launchers
// ===========================================================================
static int head_blocks(int64_t d) { return d <= 64 ? 2 : d <= 128 ? 4 : 8; }
static int dtype_terms(int32_t dt) { return dt == QAMW_F32 ? 3 : dt == QAMW_F16 ? 2 : 1; }

AttentionPlan attention_plan(int64_t T, int64_t sequences, int64_t max_queries, int64_t heads, int64_t group, int64_t d,
                             int64_t tokens, int32_t qdt, int32_t odt) {
  const int64_t most_rows = std::min(max_queries, T) * group;
  const int terms = std::max(dtype_terms(qdt), dtype_terms(odt)), db = head_blocks(d);
  AttentionPlan p;
  p.rows = 16;
  (void)terms;
  p.row_tiles = (int)std::min<int64_t>(tiles_of(most_rows, p.rows), INT32_MAX);
  const int64_t items = sequences * heads * p.row_tiles, tiles = std::max<int64_t>(tiles_of(tokens, kTileTokens), 1);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({tiles_of(4 * kCus, std::max<int64_t>(items, 1)), tiles, kMaxSplits}));
  p.groups = items * p.splits;
  p.bytes = p.splits > 1 ? (size_t)p.groups * p.rows * (32 * db + 2) * sizeof(float) : 0;
  return p;
}

template <int DB, int RT, int kTerms>
static int attention_as(const AttentionArgs& a, const AttentionPlan& p, float* part, hipStream_t st) {
  hipLaunchKernelGGL((cache_attention_kernel<DB, RT, kTerms>), dim3((unsigned)p.groups), dim3(kAttnThreads), 0, st, a,
                     p.row_tiles, p.splits, part);
  const int rc = check_launch("cache_attention_kernel");
  if (rc || p.splits == 1) return rc;
  hipLaunchKernelGGL((cache_attention_join_kernel<DB>), dim3((unsigned)tiles_of(a.T * a.c.heads * a.group, kAttnWaves)),
                     dim3(kAttnThreads), 0, st, a, p.rows, p.row_tiles, p.splits, part);
  return check_launch("cache_attention_join_kernel");
}
template <int DB>
static int attention_of(const AttentionArgs& a, const AttentionPlan& p, float* part, hipStream_t st) {
  const int terms = std::max(dtype_terms(a.qdt), dtype_terms(a.odt));
  if (terms == 3) return attention_as<DB, 1, 3>(a, p, part, st);
  if (terms == 2) return attention_as<DB, 1, 2>(a, p, part, st);
  return attention_as<DB, 1, 1>(a, p, part, st);
}
int launch_cache_attention(const AttentionArgs& a, const AttentionPlan& p, void* ws, hipStream_t st) {
  const int db = head_blocks(a.c.d);
  if (db == 2) return attention_of<2>(a, p, (float*)ws, st);
  if (db == 4) return attention_of<4>(a, p, (float*)ws, st);
  return attention_of<8>(a, p, (float*)ws, st);
}

}  // namespace qamw
