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
#include <type_traits>

#include "cache_spans.h"
#include "mx4_device.h"
#include "qamw.h"
#include "qamw_device.h"
#include "qamw_internal.h"
#include "tile_product.h"

namespace qamw {

constexpr int kAttnWaves = 4, kAttnThreads = kAttnWaves * kWave;
constexpr int kWaveTokens = 32, kTileTokens = kAttnWaves * kWaveTokens;
constexpr int kMaxSplits = 64;                     // a wavefront joins them, one a lane
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ Sequence sequence_of(const AttentionArgs& a, int b) {
  const int64_t most = (int64_t)a.cols << a.c.page_shift;
  return a.starts ? clamped_sequence(a.starts[b], a.starts[b + 1], a.T, a.lengths[b], most)
                  : clamped_sequence(b, b + 1, a.T, a.lengths[b], most);
}
// query rows of a key head that are computed: those of at most max_queries queries (T group is at most 2^30)
__device__ __forceinline__ int rows_of(const AttentionArgs& a, const Sequence& s) { return min(s.n, a.most) * a.group; }
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
  t.count = hi > lo && a.c.pages > 0 ? (hi + kTileTokens - 1) / kTileTokens - t.first : 0;
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

// the 8 four-bit elements of w times the scale, as bf16 (exact) or fp16 (exact
// where f16_holds)
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
template <bool kF16>
__device__ __forceinline__ void decode_16(uint32_t w, float s, uint32_t (&o)[4]) {
  if constexpr (kF16) {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
  } else {
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  }
}
// Scale codes of NaN blocks, and 253 and 254, which no write makes: they stand
// for values that neither bf16 nor fp32 holds all of, and their infinities
// would reach rows that must not see the token, by a weight of 0.
__device__ __forceinline__ bool is_nan_code(uint32_t code) { return code > 252u; }
// Scale codes whose blocks fp16 holds as normal numbers: 2^e / 2 to 6 2^e with e
// in [-13, 13]; a code of 0 for the zeros that have it (of values below 2^-124,
// which have it too, fp16 makes zeros).
__device__ __forceinline__ bool f16_holds(uint32_t code) { return code - 114u <= 26u || code == 0u; }
// x as a sum of kTerms bf16 numbers: 8, 16 or 24 bits of it
template <int kTerms>
__device__ __forceinline__ void split_bf16x2(float x0, float x1, uint32_t (&o)[kTerms]) {
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    o[t] = pack_bf16x2(x0, x1);
    if (t + 1 < kTerms) x0 -= __uint_as_float(o[t] << 16), x1 -= __uint_as_float(o[t] & 0xffff0000u);
  }
}
__device__ __forceinline__ f32x4 mfma_f16(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_bf16(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Workgroup -> (sequence and key head, row tile, share).  Where the pairs
// divide among the 8 XCDs, all work of a pair goes to one: its keys and values
// then pass through one L2.  The last rows, which see most tokens, first.
struct Place {
  int pair, b, h, tile, share;
};
__device__ __forceinline__ Place place_of(const AttentionArgs& a, int row_tiles, int splits) {
  const int pairs = a.sequences * a.c.heads, per = row_tiles * splits, id = blockIdx.x;
  Place p;
  int inner;
  if (pairs % 8 == 0) p.pair = id / 8 / per * 8 + id % 8, inner = id / 8 % per;
  else p.pair = id / per, inner = id % per;
  p.b = p.pair / a.c.heads, p.h = p.pair - p.b * a.c.heads;
  p.tile = row_tiles - 1 - inner / splits, p.share = inner % splits;
  return p;
}
// uniform loads of the page table go through the scalar cache
typedef const __attribute__((address_space(4))) int32_t* ConstantInts;

// One head's rows of a page, keys or values.  For a page outside the cache
// page 0 is read (there is one: without pages there are no tiles) and nothing
// of it used.
struct PageRows {
  const uint8_t *codes, *scales;                   // of page 0
  uint32_t code_step, scale_step;                  // from page to page
  uint32_t code_bytes, scale_bytes;                // of one
  __device__ __forceinline__ PageRows(const AttentionArgs& a, int kv, int h) {
    code_bytes = (uint32_t)(16 * a.c.nb) << a.c.page_shift, scale_bytes = (uint32_t)a.c.sb << a.c.page_shift;
    code_step = code_bytes * (uint32_t)a.c.heads, scale_step = scale_bytes * (uint32_t)a.c.heads;
    codes = a.codes + kv * a.c.pages * code_step + (int64_t)h * code_bytes;
    scales = a.scales + kv * a.c.pages * scale_step + (int64_t)h * scale_bytes;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t code_buffer(uint32_t page) const {
    return buffer_of(codes + (uint64_t)page * code_step, code_bytes);
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_buffer(uint32_t page) const {
    return buffer_of(scales + (uint64_t)page * scale_step, scale_bytes);
  }
};

// A lane's values of 8 tokens, 4 g + (0 .. 3) of either group of 16, as they
// lie in the cache: elements 2 DB l16 + (0 .. 2 DB - 1) of each, and the scale
// codes of all their blocks.
template <int DB>
struct RawValues {
  static constexpr int VW = DB == 8 ? 2 : 1;       // words of a token's elements in one lane
  uint32_t w[2][4][VW], s[2][DB];
  // a group's page through its two buffers, the group's rows from byte offsets c and sc of them
  __device__ __forceinline__ void load(int i, __amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales, int rb, int c, int sc,
                                       int l16, int g) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int off = (int)(l16 * DB < rb ? (uint32_t)((4 * g + e) * rb + l16 * DB) : kPastEnd);
      if constexpr (DB == 2) {
        w[i][e][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(codes, off, c, 0);
      } else if constexpr (DB == 4) {
        w[i][e][0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(codes, off, c, 0);
      } else {
        const auto x = __builtin_amdgcn_raw_buffer_load_b64(codes, off, c, 0);
        w[i][e][0] = (uint32_t)x[0], w[i][e][VW - 1] = (uint32_t)x[1];
      }
    }
    if constexpr (DB == 2) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(scales, 8 * g, sc, 0);
      s[i][0] = (uint32_t)x[0], s[i][1] = (uint32_t)x[1];
    } else {
#pragma unroll
      for (int k = 0; k < DB; k += 4) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b128(scales, 4 * DB * g + 4 * k, sc, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][k + e] = (uint32_t)x[e];
      }
    }
  }
  // codes of the 8 tokens and the scale code of this lane's block of each
  __device__ __forceinline__ void take(uint32_t (&vc)[8], uint32_t (&vw)[8][VW], int l16) const {
    const int block = l16 * DB / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (DB == 2) vc[4 * i + e] = s[i][e / 2] >> (16 * (e & 1) + 8 * block) & 255u;
        if constexpr (DB == 4) vc[4 * i + e] = s[i][e] >> (8 * block) & 255u;
        if constexpr (DB == 8) vc[4 * i + e] = (block < 4 ? s[i][2 * e] : s[i][2 * e + 1]) >> (8 * (block & 3)) & 255u;
#pragma unroll
        for (int n = 0; n < VW; ++n) vw[4 * i + e][n] = w[i][e][n];
      }
  }
};
// tokens outside [lo, hi) or of no page, which may hold anything, as 0; t: the lane's first token
template <int DB>
__device__ __forceinline__ void clear_unseen(uint32_t (&vc)[8], uint32_t (&vw)[8][RawValues<DB>::VW], int t, int lo, int hi,
                                             const bool (&ok)[2]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (t + 12 * (e / 4) + e < lo || t + 12 * (e / 4) + e >= hi || !ok[e / 4]) {
      vc[e] = 0;
#pragma unroll
      for (int n = 0; n < RawValues<DB>::VW; ++n) vw[e][n] = 0;
    }
}
// NaN blocks as 0, and where they were as 1 in bf16
template <int DB>
__device__ __forceinline__ i32x4 take_nan(uint32_t (&vc)[8], uint32_t (&vw)[8][RawValues<DB>::VW]) {
  i32x4 bad = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (is_nan_code(vc[e])) {
      bad[e / 2] |= 0x3f80 << (16 * (e & 1));
      vc[e] = 0;
#pragma unroll
      for (int n = 0; n < RawValues<DB>::VW; ++n) vw[e][n] = 0;
    }
  return bad;
}
__device__ __forceinline__ bool any_nan(const uint32_t (&vc)[8]) {
  uint32_t most = vc[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) most = max(most, vc[e]);
  return __ballot(is_nan_code(most)) != 0;
}
// The operands V^T, in fp16 or bf16: put(t, f) for the t-th element of every
// lane.  Pairs of tokens are put together by byte permutes.
template <int DB, bool kF16, class Put>
__device__ __forceinline__ void decode_values(const uint32_t (&vc)[8], const uint32_t (&vw)[8][RawValues<DB>::VW], Put&& put) {
#pragma unroll
  for (int n = 0; n < RawValues<DB>::VW; ++n) {
    uint32_t d[8][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) decode_16<kF16>(vw[e][n], __uint_as_float(vc[e] << 23), d[e]);
#pragma unroll
    for (int x = 0; x < (DB == 2 ? 2 : 4); ++x) {
      i32x4 even, odd;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        even[e] = (int)__builtin_amdgcn_perm(d[2 * e + 1][x], d[2 * e][x], 0x05040100);
        odd[e] = (int)__builtin_amdgcn_perm(d[2 * e + 1][x], d[2 * e][x], 0x07060302);
      }
      put(8 * n + 2 * x, even);
      put(8 * n + 2 * x + 1, odd);
    }
  }
}

// The reference of the exponentials follows the maximum only when a score
// exceeds it by 2^8 more than it is meant to (weights are then up to 256 times
// as large): nearly all tiles go without an exchange between lanes and without
// a pass over the sums.  It is put kLift powers of two below the maximum.
// Scores are those of 8 tokens of one row in every lane.
template <int kLift, int RT, int MT>
__device__ __forceinline__ void follow_maximum(const f32x4 (&s)[RT][2], float c, float (&m)[RT], float (&l)[RT],
                                               f32x4 (&o)[RT][MT]) {
  float top[RT];
  bool above = false;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const float x = fmaxf(fmaxf(s[j][0][0], s[j][0][1]), fmaxf(s[j][0][2], s[j][0][3])),
                y = fmaxf(fmaxf(s[j][1][0], s[j][1][1]), fmaxf(s[j][1][2], s[j][1][3]));
    top[j] = fmaxf(x, y) * c;
    above |= top[j] > m[j] + (8.0f + kLift);
  }
  if (!__ballot(above)) return;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    float x = fmaxf(top[j], __shfl_xor(top[j], 16));
    x = fmaxf(m[j], fmaxf(x, __shfl_xor(x, 32)) - kLift);
    const float f = __builtin_amdgcn_exp2f(m[j] - x);
    m[j] = x;
    l[j] *= f;
#pragma unroll
    for (int t = 0; t < MT; ++t) o[j][t] *= f;
  }
}
// the weights 2^(s c - m), put(row fragment, word of the operand P, two weights), and their sums
template <int RT, class Put>
__device__ __forceinline__ void weights(const f32x4 (&s)[RT][2], float c, const float (&m)[RT], float (&l)[RT], Put&& put) {
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i][e], c, -m[j])),
                    p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][i][e + 1], c, -m[j]));
        l[j] += p0 + p1;
        put(j, 2 * i + e / 2, p0, p1);
      }
}
// Blocks that are NaN must reach the rows that see their token and no others,
// whose weight of it is 0: the caller takes them as 0, and the elements of a
// row become NaN where the product of "sees the token" and "is NaN" (bad: 1 or
// 0 in bf16 for the lane's 8 tokens) counts any.
template <int RT, int MT, class Sees>
__device__ __forceinline__ void spread_nan(i32x4 bad, Sees&& sees, f32x4 (&o)[RT][MT]) {
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
// n elements of a row from element j
template <int n>
__device__ __forceinline__ void store_elements(int32_t dt, void* row, int j, int d, const float (&x)[n]) {
  if constexpr (n == 4) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (j + t < d) {
        if (dt == QAMW_F32) ((float*)row)[j + t] = x[t];
        else ((uint16_t*)row)[j + t] = dt == QAMW_F16 ? MemF16::put(x[t]) : MemBf16::put(x[t]);
      }
  } else {
#pragma unroll
    for (int t = 0; t < n; t += 8) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[t + e];
      store8_as(dt, row, j + t, d, y);
    }
  }
}

// wavefronts a SIMD that the registers are to allow
template <int DB, int RT, int kTerms> constexpr int attn_waves() { return DB == 8 || RT == 2 || kTerms == 3 ? 2 : 3; }
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
//     the same 8 tokens, and the m-th instruction multiplies the m-th element
//     of every lane.
//
// kTerms: q is a sum of that many bf16 numbers: 1 for bf16 in and out, 2 where
// fp16 and 3 where fp32 takes part; the weights are 2, 2 and 3 of them (each
// rounded by at most 2^-16 or 2^-24 of itself; as one number, by 2^-8, the
// error of a bf16 output grew from 0.0016 to 0.0024 in the root mean square).
// Sums are fp32 throughout.
//
// One query a sequence is bound by reading the cache: 4 sequences of up to
// 131072 tokens, 64/8 heads of 128, 98 us and 6 us to join, 518 MB, 5.05 TB/s in
// all; 64 of up to 8192, 32/8 heads, 90 us, 421 MB, 4.7 TB/s.  Two workgroups a CU
// read as fast as three or more (4 sequences: 103 us with 512 workgroups, 127 us
// with 2048).  Accumulators in the accumulation registers cost a copy for every
// use: the launch bounds keep the compiler from them (4 chunks of 2048 rows: 1.50
// ms against 1.10 ms).  A short context waits for its tiles one after another,
// 0.65 us each.
// ---------------------------------------------------------------------------
template <int DB, int RT, int kTerms>
__global__ __launch_bounds__(kAttnThreads, (attn_waves<DB, RT, kTerms>())) void cache_attention_kernel(
    AttentionArgs a, int row_tiles, int splits, float* __restrict__ part) {
  constexpr int MT = 2 * DB;                       // matrix instructions along the head
  constexpr int kWeightTerms = kTerms == 3 ? 3 : 2;
  constexpr int LD = 32 * DB + 4;                  // LDS row, off the banks' period
  __shared__ __align__(16) float joined[kAttnWaves * 16 * LD];
  __shared__ float stats[2][kAttnWaves][16];
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const Place at = place_of(a, row_tiles, splits);
  const int h = at.h;
  const Sequence seq = sequence_of(a, at.b);
  const int rows = rows_of(a, seq), r0 = at.tile * 16 * RT, r1 = min(rows, r0 + 16 * RT);
  if (r0 >= rows) return;
  const TileRange range = tile_range(a, seq, r0, r1, splits);
  if (at.share >= range.shares) return;
  const int k0 = range.first + (int)((int64_t)range.count * at.share / range.shares),
            k1 = range.first + (int)((int64_t)range.count * (at.share + 1) / range.shares);
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
    uint32_t k[2][DB], ks[2];
    RawValues<DB> v;
    bool page_ok[2];
  };
  const ConstantInts table = (ConstantInts)(uintptr_t)(a.table + at.b * a.table_pitch);
  const int rb = 16 * a.c.nb, shift = a.c.page_shift, in_page = (1 << shift) - 1;
  const PageRows key_rows(a, 0, h), value_rows(a, 1, h);
  auto pages_of = [&](int k, int (&page)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = k * kTileTokens + wave * kWaveTokens + 16 * i;
      page[i] = k < k1 && t < hi_any && t + 16 > lo_any ? table[t >> shift] : -1;
    }
  };
  const uint32_t k_at = (uint32_t)(l16 * rb + g * (4 * DB));
  const uint32_t ks_at = (uint32_t)(l16 * a.c.sb + (DB == 2 ? g >> 1 : DB == 4 ? g : 2 * g));
  auto load = [&](int k, const int (&page)[2], Raw& r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool ok = page[i] >= 0 && page[i] < a.c.pages;
      r.page_ok[i] = ok;
      const uint32_t id = ok ? (uint32_t)page[i] : 0u;
      const __amdgpu_buffer_rsrc_t bk = key_rows.code_buffer(id), bks = key_rows.scale_buffer(id);
      // offsets stay inside a page: the range check subtracts the scalar one from its size
      const int in = (k * kTileTokens + wave * kWaveTokens + 16 * i) & in_page;
      const int sc = in * rb, ss = in * a.c.sb;
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
      r.v.load(i, value_rows.code_buffer(id), value_rows.scale_buffer(id), rb, sc, ss, l16, g);
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
        decode_16<false>(r.k[i][w], __uint_as_float((DB == 8 && w < 4 ? r.ks[i] & 255u : DB == 8 ? r.ks[i] >> 8 : r.ks[i]) << 23), kd);
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
    follow_maximum<0, RT, MT>(s, c, m, l, o);
    i32x4 p[RT][kWeightTerms];
    weights<RT>(s, c, m, l, [&](int j, int at, float p0, float p1) __attribute__((always_inline)) {
      uint32_t t[kWeightTerms];
      split_bf16x2<kWeightTerms>(p0, p1, t);
#pragma unroll
      for (int n = 0; n < kWeightTerms; ++n) p[j][n][at] = (int)t[n];
    });
    uint32_t vc[8], vw[8][RawValues<DB>::VW];
    r.v.take(vc, vw, l16);
    if (!whole) {                                  // rows may see different tokens
      clear_unseen<DB>(vc, vw, t0 + 4 * g, lo_any, hi_any, r.page_ok);
      if (any_nan(vc)) spread_nan<RT, MT>(take_nan<DB>(vc, vw), sees, o);
    }
    decode_values<DB, false>(vc, vw, [&](int t, i32x4 f) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int n = 0; n < kWeightTerms; ++n) o[j][t] = mfma_bf16(f, p[j][n], o[j][t]);
    });
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
    const int sub = threadIdx.x >> 4, col = (threadIdx.x & 15) * MT, row = r0 + 16 * j + sub;
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
        const f32x4 v = *reinterpret_cast<const f32x4*>(joined + (w * 16 + sub) * LD + col + t);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t + e] += v[e];
      }
    }
    if (range.shares > 1) {
      float* to_part = part + (((int64_t)at.pair * row_tiles + at.tile) * splits + at.share) * part_floats<DB, RT>();
#pragma unroll
      for (int t = 0; t < MT; t += 4)
        *reinterpret_cast<f32x4*>(to_part + (16 * j + sub) * 32 * DB + col + t) = f32x4{x[t], x[t + 1], x[t + 2], x[t + 3]};
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
    store_elements<MT>(a.odt, row_at(a.out, a.odt, query * a.o_token + head * a.o_head), col, a.c.d, x);
    if (a.lse && (threadIdx.x & 15) == 0)
      a.lse[query * a.c.heads * a.group + head] = sum != 0.0f ? (ref + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// Many query rows: each of the 4 wavefronts has 32 rows of its own and goes
// through all tokens of the workgroup's share.  For bf16 queries and output
// and heads of up to 128 elements.
//   * Keys are decoded to bf16 in every wavefront, straight into the registers
//     of the product, for its 32 rows: scores are sums in fp32 of exact
//     products, the same as in the kernel above, whichever of the two takes a
//     call.  (As they lie in the cache, on the scaled matrix instructions with
//     a query as two 8-bit numbers, they took 596 us of the case below and now
//     648, but such an instruction sums 128 products cut off below 24 bits of
//     the largest: lse was off by 4e-5 in the root mean square where scores go
//     to 25, now 9e-7.)
//   * Values are decoded once a workgroup, each wavefront 32 tokens, into LDS
//     in the layout of the matrix operand, two tiles in turn: one barrier a
//     tile.  They and the weights go in fp16, which rounds a weight by at most
//     2^-11 of itself.  Its range is used whole: weights are up to 2^15 and a
//     row's largest at least 2^7, so that small ones are held to within 2^-25,
//     2^-32 of the largest, and 2^17 tokens that far down lose 2^-15 of the row
//     (with a largest weight of 1, those below 2^-25 of it vanished).  The
//     results of a workgroup that met a value beyond fp16 (or a NaN block) are
//     dropped, and a second launch does its work with values in bf16 and the
//     weights as two bf16 numbers.
// 4 chunks of 2048 queries behind up to 8192 tokens, 32/8 heads of 128: 648 us, 920
// TFLOP/s; 1.47 ms where every workgroup meets a value that fp16 does not hold
// (values times 2^-12).  Matrix instructions are 39 % busy; the other vector
// instructions of 32 x 32 scores, 156 with 16 exponentials and the decoding of
// the keys, take about as long as the 32 matrix ones, two wavefronts a SIMD
// overlap them in part.
// ---------------------------------------------------------------------------
template <bool kF16>
__global__ __launch_bounds__(kAttnThreads, 2) void cache_attention_chunk_kernel(AttentionArgs a, int row_tiles, int splits,
                                                                                float* __restrict__ part, int* __restrict__ redo) {
  constexpr int DB = 4, RT = 2, MT = 2 * DB, kWaveRows = 16 * RT, kRows = kAttnWaves * kWaveRows;
  __shared__ __align__(16) i32x4 staged[2][kAttnWaves][MT][kWave];
  __shared__ __align__(16) i32x4 staged_bad[2][kAttnWaves][kWave];
  __shared__ int staged_nan[2][kAttnWaves], unfit;
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (kF16) {
    if (threadIdx.x == 0) redo[blockIdx.x] = 0, unfit = 0;
    __syncthreads();
  } else if (!redo[blockIdx.x]) {
    return;
  }
  const Place at = place_of(a, row_tiles, splits);
  const int h = at.h;
  const Sequence seq = sequence_of(a, at.b);
  const int rows = rows_of(a, seq), r0 = at.tile * kRows, r1 = min(rows, r0 + kRows);
  if (r0 >= rows) return;
  const TileRange range = tile_range(a, seq, r0, r1, splits);
  if (at.share >= range.shares) return;
  const int k0 = range.first + (int)((int64_t)range.count * at.share / range.shares),
            k1 = range.first + (int)((int64_t)range.count * (at.share + 1) / range.shares);
  // tokens that any row of the workgroup sees; that any and every row of the wavefront sees
  const int lo_group = span_begin(a, seq, r0 / a.group), hi_group = span_end(a, seq, (r1 - 1) / a.group);
  const int w0 = r0 + wave * kWaveRows, w1 = min(rows, w0 + kWaveRows);
  const int last = max(w1 - 1, 0) / a.group, first = min(w0, rows - 1) / a.group;
  const int lo_any = span_begin(a, seq, first), hi_any = w0 < rows ? span_end(a, seq, last) : 0;
  const int lo_all = span_begin(a, seq, last), hi_all = span_end(a, seq, first);

  // ---- queries: lane group g holds block g of a row's elements, as it does of the keys
  i32x4 q[RT][DB];
  int row_lo[RT], row_hi[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int row = min(w0 + 16 * j + l16, rows - 1), i = row / a.group, head = h * a.group + row % a.group;
    row_lo[j] = span_begin(a, seq, i), row_hi[j] = span_end(a, seq, i);
    const void* p = row_at(a.Q, QAMW_BF16, (seq.first + i) * a.q_token + head * a.q_head);
#pragma unroll
    for (int w = 0; w < DB; ++w) {
      float x[8];
      load8<MemBf16>((const uint16_t*)p, 8 * (g * DB + w), a.c.d, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) q[j][w][e] = (int)pack_bf16x2(x[2 * e], x[2 * e + 1]);
    }
  }

  f32x4 o[RT][MT] = {};
  float m[RT], l[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) m[j] = -FLT_MAX, l[j] = 0.0f;

  const ConstantInts table = (ConstantInts)(uintptr_t)(a.table + at.b * a.table_pitch);
  const int rb = 16 * a.c.nb, shift = a.c.page_shift, in_page = (1 << shift) - 1;
  const PageRows key_rows(a, 0, h), value_rows(a, 1, h);

  // ---- keys, 16 tokens after 16: a lane holds block g of token l % 16.  The
  // page's buffers change where a page ends; the next one's number is read then.
  struct Keys {
    i32x4 c[2];
    int s[2];
    bool ok[2];
  };
  __amdgpu_buffer_rsrc_t key_codes, key_scales;
  bool key_ok = false;
  int next_page = -1;
  auto turn_page = [&](int t) __attribute__((always_inline)) {
    key_ok = next_page >= 0 && next_page < a.c.pages;
    const uint32_t id = key_ok ? (uint32_t)next_page : 0u;
    key_codes = key_rows.code_buffer(id), key_scales = key_rows.scale_buffer(id);
    next_page = table[min((t >> shift) + 1, a.cols - 1)];
  };
  const int kc_at = g < a.c.nb ? l16 * rb + 16 * g : (int)kPastEnd, ks_at = g < a.c.nb ? l16 * a.c.sb + g : (int)kPastEnd;
  auto load_keys = [&](int t0, Keys& r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int in = (t0 + 16 * i) & in_page;
      if (in == 0) turn_page(t0 + 16 * i);
      r.ok[i] = key_ok;
      r.c[i] = load16(key_codes, (uint32_t)kc_at, (uint32_t)(in * rb));
      r.s[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(key_scales, ks_at, in * a.c.sb, 0);
    }
  };

  // ---- values of this wavefront's 32 tokens of a tile, raw, then as operands in LDS
  RawValues<DB> raw;
  bool raw_ok[2];
  int page[2];
  auto value_pages = [&](int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) page[i] = table[min((k * kTileTokens + wave * kWaveTokens + 16 * i) >> shift, a.cols - 1)];
  };
  auto load_values = [&](int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      raw_ok[i] = page[i] >= 0 && page[i] < a.c.pages;
      const uint32_t id = raw_ok[i] ? (uint32_t)page[i] : 0u;
      const int in = (k * kTileTokens + wave * kWaveTokens + 16 * i) & in_page;
      raw.load(i, value_rows.code_buffer(id), value_rows.scale_buffer(id), rb, in * rb, in * a.c.sb, l16, g);
    }
  };
  auto stage_values = [&](int k) __attribute__((always_inline)) {
    const int t0 = k * kTileTokens + wave * kWaveTokens;
    uint32_t vc[8], vw[8][RawValues<DB>::VW];
    raw.take(vc, vw, l16);
    if (t0 < lo_group || t0 + kWaveTokens > hi_group || !raw_ok[0] || !raw_ok[1])
      clear_unseen<DB>(vc, vw, t0 + 4 * g, lo_group, hi_group, raw_ok);
    if constexpr (kF16) {
      bool fits = true;
#pragma unroll
      for (int e = 0; e < 8; ++e) fits &= f16_holds(vc[e]);
      if (!fits) unfit = 1;
    } else {
      const bool nan = any_nan(vc);
      if (nan) staged_bad[k & 1][wave][lane] = take_nan<DB>(vc, vw);
      if (lane == 0) staged_nan[k & 1][wave] = nan;
    }
    decode_values<DB, kF16>(vc, vw, [&](int t, i32x4 f) __attribute__((always_inline)) { staged[k & 1][wave][t][lane] = f; });
  };

  const float c = a.scale * kLog2e;
  auto multiply_keys = [&](const Keys& r, f32x4 (&s)[RT][2]) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < DB; ++w)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t kd[4];
        decode_16<false>((uint32_t)r.c[i][w], __uint_as_float((uint32_t)r.s[i] << 23), kd);
        const i32x4 kf = {(int)kd[0], (int)kd[1], (int)kd[2], (int)kd[3]};
#pragma unroll
        for (int j = 0; j < RT; ++j) s[j][i] = mfma_bf16(kf, q[j][w], w ? s[j][i] : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      }
  };
  auto compute = [&](int k, int sub, f32x4 (&s)[RT][2], const bool (&ok)[2]) __attribute__((always_inline)) {
    const int t0 = k * kTileTokens + sub * kWaveTokens;
    if (t0 >= hi_any || t0 + kWaveTokens <= lo_any) return;
    const bool whole = t0 >= lo_all && t0 + kWaveTokens <= hi_all && ok[0] && ok[1];
    auto sees = [&](int j, int i, int e) __attribute__((always_inline)) {
      const int t = t0 + 16 * i + 4 * g + e;
      return t >= row_lo[j] && t < row_hi[j] && ok[i];
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
    follow_maximum<kF16 ? 7 : 0, RT, MT>(s, c, m, l, o);
    // the values are on their way from LDS while the weights are made
    constexpr int kWeightTerms = kF16 ? 1 : 2;
    i32x4 v[MT], p[RT][kWeightTerms];
#pragma unroll
    for (int t = 0; t < MT; ++t) v[t] = staged[k & 1][sub][t][lane];
    __builtin_amdgcn_sched_barrier(0);
    weights<RT>(s, c, m, l, [&](int j, int at, float p0, float p1) __attribute__((always_inline)) {
      if constexpr (kF16) {
        const f32x2_t both = {p0, p1};
        p[j][0][at] = __builtin_bit_cast(int, __builtin_convertvector(both, f16x2_t));
      } else {
        uint32_t t[2];
        split_bf16x2<2>(p0, p1, t);
        p[j][0][at] = (int)t[0], p[j][kWeightTerms - 1][at] = (int)t[1];
      }
    });
    if constexpr (!kF16)
      if (__builtin_amdgcn_readfirstlane(staged_nan[k & 1][sub])) spread_nan<RT, MT>(staged_bad[k & 1][sub][lane], sees, o);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int n = 0; n < kWeightTerms; ++n)
          o[j][t] = kF16 ? mfma_f16(v[t], p[j][n], o[j][t]) : mfma_bf16(v[t], p[j][n], o[j][t]);
  };

  if (k0 < k1) {
    Keys keys;
    f32x4 s[2][RT][2];
    bool ok[2][2];
    value_pages(k0);
    next_page = table[(k0 * kTileTokens) >> shift];
    if ((k0 * kTileTokens) & in_page) turn_page(k0 * kTileTokens);       // the share starts inside a page
    load_keys(k0 * kTileTokens, keys);
    load_values(k0);
    value_pages(k0 + 1);
    multiply_keys(keys, s[0]);
    ok[0][0] = keys.ok[0], ok[0][1] = keys.ok[1];
    load_keys(k0 * kTileTokens + kWaveTokens, keys);
    stage_values(k0);
    load_values(k0 + 1);
    __syncthreads();
    // Tile k is multiplied from one half of LDS while the other, which nobody
    // reads since the last barrier, is filled.  The scores of the next 32
    // tokens are under way in the matrix cores while the weights of these are made.
    for (int k = k0; k < k1; ++k) {
#pragma unroll
      for (int sub = 0; sub < 4; ++sub) {
        multiply_keys(keys, s[~sub & 1]);
        ok[~sub & 1][0] = keys.ok[0], ok[~sub & 1][1] = keys.ok[1];
        load_keys(k * kTileTokens + (sub + 2) * kWaveTokens, keys);
        if (sub == 0) value_pages(k + 2);
        compute(k, sub, s[sub & 1], ok[sub & 1]);
        if (sub == 1) {
          stage_values(k + 1);
          load_values(k + 2);
        }
      }
      __syncthreads();
    }
  }

  // The last barrier has passed, nobody sets the flag any more.  (Looked at
  // inside the loop it makes the compiler spill: 620 us became 850.)
  if constexpr (kF16)
    if (unfit) {
      if (threadIdx.x == 0) redo[blockIdx.x] = 1;
      return;
    }

  // ---- results: lane l has row l % 16 and elements MT (4 (l / 16) + e) + t
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    l[j] += __shfl_xor(l[j], 16);
    l[j] += __shfl_xor(l[j], 32);
    const int row = w0 + 16 * j + l16;
    if (row >= rows) continue;
    if (range.shares > 1) {
      float* to = part + (((int64_t)at.pair * row_tiles + at.tile) * splits + at.share) * ((int64_t)kRows * (32 * DB + 2));
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int t = 0; t < MT; t += 4)
          *reinterpret_cast<f32x4*>(to + (row - r0) * 32 * DB + MT * (4 * g + e) + t) =
              f32x4{o[j][t][e], o[j][t + 1][e], o[j][t + 2][e], o[j][t + 3][e]};
      if (g == 0) {
        to[kRows * 32 * DB + row - r0] = m[j];
        to[kRows * (32 * DB + 1) + row - r0] = l[j];
      }
      continue;
    }
    const int64_t query = seq.first + row / a.group;
    const int head = h * a.group + row % a.group;
    const float inv = l[j] != 0.0f ? 1.0f / l[j] : 0.0f;
    void* to = row_at(a.out, QAMW_BF16, query * a.o_token + head * a.o_head);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) x[t] = o[j][t][e] * inv;
      store_elements<MT>(QAMW_BF16, to, MT * (4 * g + e), a.c.d, x);
    }
    if (a.lse && g == 0)
      a.lse[query * a.c.heads * a.group + head] = l[j] != 0.0f ? (m[j] + __builtin_amdgcn_logf(l[j])) * kLn2 : -INFINITY;
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
  const int64_t row = (query - seq.first) * a.group + (head - h * a.group);
  if (query < seq.first || row >= rows_of(a, seq)) return;
  const int tile = (int)(row / tile_rows), r0 = tile * tile_rows, r1 = min(rows_of(a, seq), r0 + tile_rows);
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
  for (int s0 = 0; s0 < range.shares; s0 += 8) {   // eight shares' rows in flight; past the last one that again, not added
    float v[8][E];
#pragma unroll
    for (int s = 0; s < 8; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) v[s][e] = p[min(s0 + s, range.shares - 1) * floats + at * 32 * DB + E * lane + e];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const float fs = __shfl(f, min(s0 + s, range.shares - 1));
      if (s0 + s < range.shares)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += fs * v[s][e];
    }
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

// Fragments of 16 query rows a workgroup takes.  8 is the kernel of many rows:
// heads of 65 to 128 elements in bf16, from 1024 rows a key head on, where its
// 128 rows a workgroup leave enough workgroups (8 sequences of up to 4096 tokens,
// 32/8 heads of 128: 1024 rows 145 us against 168 us with 2 fragments, 512 rows
// 104 us and 100 us; heads of 64 would fill half its instructions).  2 fragments
// share the decoding (256 rows 52 us, with 1 fragment 60 us; 64 rows 28 and 30
// us, in one sequence of 8192 tokens 19 and 17 us); their registers allow them
// for bf16 and heads of up to 128 elements.
static int row_fragments(int64_t rows, int db, int terms) {
  if (terms > 1 || db == 8 || rows <= 128) return 1;
  return db == 4 && rows > 768 ? 8 : 2;
}

// Into how many shares the tokens of an item go: rounds of workgroups (two a
// CU: more of them at a time read no faster) times the tiles of a share, and
// what joining costs.  Times of a tile of 128 tokens in a round, microseconds;
// an item of up to 12 tiles in one share takes no longer than two launches (1
// sequence of 1000 tokens, 32 heads: 11.1 us against 10.7 us in 8 shares).  No
// share is longer than 96 tiles, however many items there are: they may be uneven.
static int shares_of(int64_t items, int64_t tiles, int rows) {
  if (tiles <= 12) return 1;
  const double tile_us = rows == 16 ? 0.65 : rows == 32 ? 0.9 : 2.7;
  double best_us = 1e30;
  int best = 1;
  for (int64_t s = tiles_of(tiles, 96); s <= kMaxSplits && s <= tiles / 2; ++s) {
    const double us = (double)tiles_of(items * s, 2 * kCus) * (double)tiles_of(tiles, s) * tile_us + (s > 1 ? 5.0 + 0.1 * (double)s : 0.0);
    if (us < 0.97 * best_us) best_us = us, best = (int)s;
  }
  return tiles_of(tiles, 96) > kMaxSplits ? kMaxSplits : best;
}

AttentionPlan attention_plan(int64_t T, int64_t sequences, int64_t max_queries, int64_t heads, int64_t group, int64_t d,
                             int64_t tokens, int32_t qdt, int32_t odt) {
  const int64_t most_rows = std::min(max_queries, T) * group;
  const int terms = std::max(dtype_terms(qdt), dtype_terms(odt)), db = head_blocks(d);
  AttentionPlan p;
  p.rows = 16 * row_fragments(most_rows, db, terms);
  p.row_tiles = (int)std::min<int64_t>(tiles_of(most_rows, p.rows), INT32_MAX);
  const int64_t items = sequences * heads * p.row_tiles, tiles = std::max<int64_t>(tiles_of(tokens, kTileTokens), 1);
  p.splits = shares_of(items, tiles, p.rows);
  p.groups = items * p.splits;
  p.bytes = p.splits > 1 ? (size_t)p.groups * p.rows * (32 * db + 2) * sizeof(float) : 0;
  if (p.rows == 128) p.bytes += (size_t)p.groups * sizeof(int);        // which workgroups gave fp16 up
  return p;
}

template <int DB>
static int join_shares(const AttentionArgs& a, const AttentionPlan& p, const float* part, hipStream_t st) {
  if (p.splits == 1) return QAMW_OK;
  hipLaunchKernelGGL((cache_attention_join_kernel<DB>), dim3((unsigned)tiles_of(a.T * a.c.heads * a.group, kAttnWaves)),
                     dim3(kAttnThreads), 0, st, a, p.rows, p.row_tiles, p.splits, part);
  return check_launch("cache_attention_join_kernel");
}
template <int DB, int RT, int kTerms>
static int attention_as(const AttentionArgs& a, const AttentionPlan& p, float* part, hipStream_t st) {
  hipLaunchKernelGGL((cache_attention_kernel<DB, RT, kTerms>), dim3((unsigned)p.groups), dim3(kAttnThreads), 0, st, a,
                     p.row_tiles, p.splits, part);
  const int rc = check_launch("cache_attention_kernel");
  return rc ? rc : join_shares<DB>(a, p, part, st);
}
static int attention_chunk(const AttentionArgs& a, const AttentionPlan& p, float* part, hipStream_t st) {
  int* redo = (int*)((char*)part + p.bytes) - p.groups;
  hipLaunchKernelGGL(cache_attention_chunk_kernel<true>, dim3((unsigned)p.groups), dim3(kAttnThreads), 0, st, a, p.row_tiles,
                     p.splits, part, redo);
  int rc = check_launch("cache_attention_chunk_kernel");
  if (rc) return rc;
  hipLaunchKernelGGL(cache_attention_chunk_kernel<false>, dim3((unsigned)p.groups), dim3(kAttnThreads), 0, st, a, p.row_tiles,
                     p.splits, part, redo);
  rc = check_launch("cache_attention_chunk_kernel");
  return rc ? rc : join_shares<4>(a, p, part, st);
}
template <int DB>
static int attention_of(const AttentionArgs& a, const AttentionPlan& p, float* part, hipStream_t st) {
  const int terms = std::max(dtype_terms(a.qdt), dtype_terms(a.odt));
  if constexpr (DB == 4)
    if (p.rows == 128) return attention_chunk(a, p, part, st);
  if constexpr (DB <= 4)
    if (p.rows == 32) return attention_as<DB, 2, 1>(a, p, part, st);
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
