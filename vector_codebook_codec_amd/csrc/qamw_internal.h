// Host-side interfaces shared by the translation units of libqamw.so:
// launch helpers of each stage, argument checks and error reporting.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qamw.h"

namespace qamw {

constexpr int kBlockThreads = 256;                   // 4 wavefronts per workgroup (most kernels)
constexpr int kWavesPerBlock = kBlockThreads / 64;
constexpr int kCalibRowsPerTile = 16;                // rows per amplitude partial sum
constexpr int kRmsRowsPerTile = 64;                  // activation rows per channel-RMS partial sum
constexpr int kOutputErrorTokens = 128;              // tokens per output-error workgroup
constexpr int kOutputErrorRows = 128;                // weight rows per output-error workgroup
constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr size_t kNoAllocScratchBytes = size_t(1) << 20;   // per-GPU workspace of qamw_encode_noalloc

// ---- errors (the message of the calling thread's last failure)
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int check_launch(const char* what);

// ---- small helpers
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
__host__ __device__ inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int elem_size(int32_t dt) { return dt == QAMW_F32 ? 4 : (dt == QAMW_BF16 || dt == QAMW_F16) ? 2 : 0; }
// rows of ld elements of a known type start 16 bytes apart (no product: ld may be of any value)
inline bool rows_aligned16(int64_t ld, int32_t dt) { return ld % (16 / elem_size(dt)) == 0; }
// Rows per calibration tile (one amplitude partial sum each).  Rows of 5 to
// 16 windows of 1024 columns are calibrated by one workgroup per CU (one
// wavefront per window), so more than kCalibTileTarget tiles would run in a
// second, mostly idle round of workgroups: there a tile grows to
// ceil(N / kCalibTileTarget) rows, a multiple of 4.  Every entry point takes
// its tiles from this one rule, so the fp32 partial sums, and sigma, agree
// bit for bit between them.
constexpr int64_t kCalibTileTarget = 256;
inline int calib_rows_per_tile(int64_t N, int64_t d) {
  const int64_t nwin = (d / 16 + 63) / 64;
  if (nwin <= 4 || nwin > 16) return kCalibRowsPerTile;
  const int64_t t = (N + kCalibTileTarget - 1) / kCalibTileTarget;
  return t <= kCalibRowsPerTile ? kCalibRowsPerTile : (int)((t + 3) / 4 * 4);
}
inline size_t calib_tiles(int64_t N, int64_t d) {
  const int64_t r = calib_rows_per_tile(N, d);
  return (size_t)((N + r - 1) / r);
}
inline unsigned grid_for_waves(int64_t waves) { return (unsigned)((waves + kWavesPerBlock - 1) / kWavesPerBlock); }

// Call Launch<L>::run(args...) for the Hadamard block size 2^L, 2 <= b <= 1024.
template <template <int> class Launch, typename... A>
int dispatch_L(int L, A&&... args) {
  switch (L) {
    case 1: return Launch<1>::run(args...);
    case 2: return Launch<2>::run(args...);
    case 3: return Launch<3>::run(args...);
    case 4: return Launch<4>::run(args...);
    case 5: return Launch<5>::run(args...);
    case 6: return Launch<6>::run(args...);
    case 7: return Launch<7>::run(args...);
    case 8: return Launch<8>::run(args...);
    case 9: return Launch<9>::run(args...);
    case 10: return Launch<10>::run(args...);
    default: return fail(QAMW_EUNSUPPORTED, "block size");
  }
}

// ---- nearest-centroid search plan (see plan.hip): a grid over [-kPlanR, kPlanR)^2
// and a coarse outer grid over [-kPlanR2, kPlanR2)^2, both centred on the origin.
// For K <= kLdsMaxK the inner grid is a table the encode kernel keeps in LDS
// (non-uniform cells, one 16-bit entry per cell, shared candidate lists); for
// larger K it is a uniform grid of per-cell records read from global memory.
constexpr int kPlanG = 512;                  // global inner grid (K > kLdsMaxK): cells per axis
constexpr float kPlanR = 5.0f;
constexpr int kPlanG2 = 128;                 // outer grid: cells per axis over [-kPlanR2, kPlanR2)
constexpr float kPlanR2 = 20.0f;
constexpr size_t kPlanHeaderBytes = 256;
constexpr size_t kPlanHeaderKOffset = 16;    // int32 K inside the header (plan.hip)
__host__ __device__ inline int plan_lmax(int K) { return K <= 2048 ? 8 : 16; }

// LDS table geometry.  Both axes share one map from kLdsBins equal bins over
// [-kPlanR, kPlanR) to cell coordinates; cells are whole runs of bins, widest
// far from the origin where centroids are sparse.  The plan's image is
// [bin -> cell map, u8 x kLdsBins][cell entries, u16 x G x G, padded to 16
// bytes][candidate lists, 4 x u16 each, lists_cap of them]; the encode kernel
// stages it into LDS in a layout of its own (below), and lists_cap is what
// fits there.
constexpr int kLdsMaxK = 2048;
constexpr int kLdsBins = 2048;
constexpr int kLdsMaxG = 255;                // the guard cell index G fits the u8 map
constexpr int kLdsThreads = 1024;            // one 16-wavefront workgroup per CU
constexpr int kLdsWaves = kLdsThreads / 64;
constexpr size_t kLdsBudget = 160 * 1024 - 1024;   // LDS bytes one encode workgroup may take
constexpr uint16_t kLdsScanAll = 0xFFFFu;    // cell entry: search the whole codebook
// The encode kernel's own LDS copy of the table: the map with one guard bin
// at each end (padded to 16 bytes), then the codebook (-cx, -cy) at 8 bytes
// per centroid, then the cells as a (G + 1) x (G + 1) array with a "scan all"
// guard row and column, then the records, then 16 packing stages.
constexpr size_t kLdsMapBytes = (kLdsBins + 2 + 15) / 16 * 16;
__host__ __device__ inline size_t lds_cell_bytes(int G) { return ((size_t)2 * (G + 1) * (G + 1) + 15) / 16 * 16; }
struct LdsGeometry {
  int G;                         // cells per axis (<= kLdsMaxG)
  int lists_cap;                 // list records the image holds
  size_t cells_off, lists_off;   // byte offsets inside the image
  size_t image_bytes;            // multiple of 16
  size_t stage_bytes;            // per-wavefront packing stage (64 B bytes)
  uint16_t edges[kLdsMaxG + 1];  // cell c covers bins [edges[c], edges[c + 1])
};
bool lds_geometry(int K, LdsGeometry* g);    // false when K > kLdsMaxK
inline bool plan_has_lds(int K) { return K >= 2 && K <= kLdsMaxK; }
size_t plan_outer_offset(int K);             // outer grid records
size_t plan_image_offset(int K);             // LDS image (K <= kLdsMaxK)
size_t plan_scratch_offset(int K);           // construction scratch (K <= kLdsMaxK)
size_t plan_bytes(int K);

// ---- stage launchers (enqueue on `st`, return a qamw_status)
int launch_scale(const float* r, float alpha, uint64_t seed, int d, float* s, float* f, hipStream_t st);
int launch_rownorm(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* s, double* rho,
                   uint16_t* rho_f16, hipStream_t st);
int launch_amplitude(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* f, const double* rho,
                     float* partial, hipStream_t st);
int launch_norm_amplitude(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* s,
                          const float* f, double* rho, uint16_t* rho_f16, float* partial, hipStream_t st);
int launch_sigma(const float* partial, int ntiles, int half_d, int N, float* sigma, float* isig, hipStream_t st);
int launch_encode_prepare(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* s, const float* sigma,
                          uint64_t seed, double* rho, uint16_t* rho_f16, float* f, float* isig, hipStream_t st);
int launch_encode(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* f, const float* isig,
                  const float* cb, int K, int B, int row_words, const double* rho, const void* plan, uint32_t* packed,
                  hipStream_t st);
int launch_encode_polar(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* f,
                        const float* isig, const float* levels, int Ka, const float* dirs, int Kp, int B,
                        int row_words, const double* rho, uint32_t* packed, hipStream_t st);
int launch_build_plan(const float* cb, int K, void* plan, hipStream_t st);
constexpr int kLloydMaxParts = 4096;                 // workgroups (fp64 partial sums) of one refinement round
int launch_lloyd_update(int L, const void* W, int32_t wdt, int N, int d, int64_t ldw, const float* f,
                        const float* isig, const double* rho, const uint32_t* packed, int row_words, int B,
                        const float* cb, int K, float* cb_out, double* distortion, unsigned long long* gacc,
                        double* partial, hipStream_t st);
int launch_channel_rms(const void* X, int32_t xdt, int T, int d, int64_t ldx, float* r, float* partial,
                       hipStream_t st);
int launch_output_error(const void* X, int32_t xdt, int T, int d, int64_t ldx, const void* W, int32_t wdt, int N,
                        int64_t ldw, const void* Wh, int32_t hdt, int64_t ldh, double* out, double* partial,
                        uint16_t* dWb, uint16_t* Xb, hipStream_t st);
int launch_rotate_act(int L, const void* X, int32_t xdt, int T, int d, int64_t ldx, const float* s, uint64_t seed,
                      uint16_t* Xr, int64_t ldr, hipStream_t st);
int launch_decode_matmul(const uint16_t* Xr, int T, int d, int64_t ldr, const uint32_t* packed, int row_words,
                         const uint16_t* rn, int N, const float* sigma, const float* cb, int K, int B, void* Y,
                         int32_t ydt, int64_t ldy, hipStream_t st);
int launch_decode(int L, const uint32_t* packed, const uint16_t* rho_f16, int N, int d, const float* s,
                  const float* sigma, uint64_t seed, const float* cb, int K, int B, int row_words, void* out,
                  int32_t odt, int64_t ldo, hipStream_t st);

// ---- microscaled 4-bit operands (mxfp4.hip): blocks of 32, 16 bytes of codes and one scale code each;
// scale rows are padded to whole 16-byte groups
constexpr int kMx4Block = 32;
inline int64_t mx4_blocks(int64_t d) { return (d + kMx4Block - 1) / kMx4Block; }
inline int64_t mx4_scale_bytes(int64_t d) { return (mx4_blocks(d) + 15) / 16 * 16; }
int launch_mx4_quantize(const void* W, int32_t wdt, int64_t N, int d, int64_t ldw, uint8_t* codes, uint8_t* scales,
                        void* values, int32_t vdt, int64_t ldv, hipStream_t st);
int launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t N, int d, void* W, int32_t odt,
                          int64_t ldo, hipStream_t st);
bool mx4_grid_fits(int64_t T, int64_t N, int64_t d);
size_t mx4_matmul_workspace_bytes(int64_t T, int64_t N, int64_t d);
// Low-rank adapters beside the product (mx4_adapter.h).  U = f_i A_i X has rows
// of `pitch` elements, the rank rounded up to 32, and lies in the workspace as
// `parts` fp32 matrices to be added (not yet times f_i), and for the product's
// tiles also as three bf16 ones.  A and B are 16-byte aligned.
constexpr int kMostAdapterParts = 4;
struct Adapters {
  const void* B;
  const int32_t* index;            // [T]; outside [0, n): none
  const float* factors;            // NULL: 1
  int n, rank, pitch, parts;
  float* u_parts;
  uint16_t* u16;                   // where the tiles multiply U and B themselves
  float* delta;                    // where adapters_in_delta: the adapters' part of Y, rows of delta_pitch
  int64_t delta_pitch;
};
bool adapters_in_delta(int64_t T, int64_t N, int32_t dt, int64_t rank);
int launch_mx4_matmul(const void* X, int32_t xdt, int64_t T, int d, int64_t ldx, const uint8_t* wcodes,
                      const uint8_t* wscales, int64_t N, void* Y, int32_t ydt, int64_t ldy, void* ws,
                      const Adapters* ad, hipStream_t st);       // ad: of X's type, or NULL
size_t adapter_workspace_bytes(int64_t T, int64_t N, int64_t d, int32_t dt, int64_t rank);
bool adapter_grid_fits(int64_t T, int64_t N, int64_t rank);
// U of X into the workspace; completes ad
int launch_adapter_shrink(const void* X, int32_t xdt, int64_t T, int64_t N, int64_t d, int64_t ldx, const void* A, void* ws,
                          Adapters* ad, hipStream_t st);
int launch_adapter_expand(int32_t dt, int64_t T, int64_t N, const Adapters& ad, hipStream_t st);

// ---- attention cache in microscaled 4 bits (cache.hip, cache_attention.hip)
struct CacheShape {
  int64_t pages;
  int heads, page_shift;           // page = 1 << page_shift tokens
  int d, nb, sb;                   // blocks of a head, bytes of a row of scales
};
constexpr int kCacheMaxHeadDim = 256;
constexpr int64_t kCacheMinPage = 16, kCacheMaxPage = 65536;
inline int cache_scale_bytes(int64_t d) { return mx4_blocks(d) <= 2 ? 2 : mx4_blocks(d) <= 4 ? 4 : 8; }
int launch_cache_write(const void* K, const void* V, int32_t dt, int64_t T, int64_t kt, int64_t kh, int64_t vt, int64_t vh,
                       const CacheShape& c, const int64_t* slots, uint8_t* codes, uint8_t* scales, hipStream_t st);
int launch_cache_read(void* K, void* V, int32_t dt, int64_t T, int64_t kt, int64_t kh, int64_t vt, int64_t vh,
                      const CacheShape& c, const int64_t* slots, const uint8_t* codes, const uint8_t* scales, hipStream_t st);

// Queries, outputs and sequences of an attention call (cache_attention.hip).
struct AttentionArgs {
  CacheShape c;
  const uint8_t *codes, *scales;
  const void* Q;
  void* out;
  float* lse;                                     // [T][group heads], or NULL
  int32_t qdt, odt;
  int64_t q_token, q_head, o_token, o_head;       // strides in elements
  const int32_t *starts, *lengths, *table;        // starts: NULL for one query a sequence
  int64_t table_pitch;
  int64_t T;
  int sequences, group, cols, most;               // most: queries of a sequence that are computed
  float scale;
  int causal, window;                             // window 0: none
};
// How the work of a call is cut: a workgroup takes `rows` query rows (query
// by head of a group) of one sequence and key head, and one of `splits` shares
// of their tokens.
struct AttentionPlan {
  int rows, row_tiles, splits;
  int64_t groups;                                 // workgroups
  size_t bytes;                                   // partial results
};
AttentionPlan attention_plan(int64_t T, int64_t sequences, int64_t max_queries, int64_t heads, int64_t group, int64_t d,
                             int64_t tokens, int32_t qdt, int32_t odt);
int launch_cache_attention(const AttentionArgs& a, const AttentionPlan& p, void* ws, hipStream_t st);

// ---- how a product [M][N] is cut into square tiles (tile_product.h).
// The measured time of one K step (128 bytes of every row), in microseconds,
// where every CU has L tiles of a shape to work on, for L = 1, 2 and per tile
// beyond (M = 16 and N = 16 L tiles, 2048 to 8192 columns).  Small tiles
// share a CU; they are for products that have too few large ones.  Shape 0
// keeps four K steps of a 64 x 64 tile in LDS instead of two, for products
// that wait for memory (64 x 32000 x 4096 in bf16: 63 us against 72 us); only
// two of its workgroups fit a CU.  fp32 products do not use it: they wait for
// the matrix instructions.  Nor do they use 256 x 256 tiles, whose registers
// leave no room for a second sum (OpF32::kChainSteps): in one chain these
// took 7.47 us a step where four 128 x 128 tiles take 7.56.
enum ProductType { kProductBf16, kProductF32, kProductMx4 };
constexpr int kCus = 256, kShapes = 4;
constexpr int kShapeTile[kShapes] = {64, 64, 128, 256};
constexpr float kNever = 1e9f;
constexpr float kShapeStepUs[3][kShapes][3] = {
    {{0.43f, 0.45f, kNever}, {0.51f, 0.51f, 0.19f}, {0.74f, 0.98f, 0.49f}, {1.60f, 3.15f, 1.58f}},
    {{kNever, kNever, kNever}, {0.62f, 1.09f, 0.50f}, {2.02f, 3.79f, 1.89f}, {kNever, kNever, kNever}},
    {{0.38f, 0.55f, kNever}, {0.45f, 0.64f, 0.24f}, {0.92f, 1.27f, 0.60f}, {1.98f, 3.84f, 1.91f}}};
inline int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }
inline double step_us(ProductType t, int shape, int64_t load) {
  const float* f = kShapeStepUs[t][shape];
  return load <= 0 ? 0.0 : load <= 2 ? f[load - 1] : f[2] * (double)load > f[1] ? f[2] * (double)load : f[1];
}
inline int64_t shape_tiles(int shape, int64_t M, int64_t N) {
  return tiles_of(M, kShapeTile[shape]) * tiles_of(N, kShapeTile[shape]);
}
inline int shape_threads(int shape) { return kShapeTile[shape] == 64 ? 256 : 512; }
// a launch is of fewer than 2^32 threads along x
inline bool grid_holds(int64_t workgroups, int threads) { return workgroups < (int64_t(1) << 32) / threads; }
// writing and reading fp32 partial results at 4 TB/s, and the launch that adds them
inline double partials_us(double elements) { return 3.0 + elements * 8e-6 / 4.0; }

struct ProductPlan {
  int shape;
  int splits;                      // along K, of every tile: as many fp32 results, added later
};
inline ProductPlan product_plan(ProductType t, int64_t M, int64_t N, int64_t steps, int most_splits) {
  ProductPlan best = {0, 1};
  double best_us = 1e30;
  for (int s = 1; s <= most_splits; ++s) {
    if (s > 1 && steps < 4 * s) break;                 // at least 4 steps a workgroup
    for (int shape = kShapes - 1; shape >= 0; --shape) {
      const double us = step_us(t, shape, tiles_of(shape_tiles(shape, M, N) * s, kCus)) * (double)tiles_of(steps, s) +
                        (s > 1 ? partials_us((double)s * M * N) : 0.0);
      if (us < 0.98 * best_us) best_us = us, best = {shape, s};
    }
  }
  return best;
}

// For a result that is written once: `whole` tiles run over all of K; the
// rest, too few to give every CU one more, are split along K.  (As smaller
// tiles in a launch of their own they took longer than the round that they
// save: the call at T = 8192, 11008 x 4096 264 us against 259 us.)
struct TailPlan {
  int shape;
  int64_t whole;
  int splits;                      // of each tile past `whole`
};
inline TailPlan tail_plan(ProductType t, int64_t M, int64_t N, int64_t steps) {
  TailPlan best = {0, 0, 1};
  double best_us = 1e30;
  for (int shape = kShapes - 1; shape >= 0; --shape) {
    const int64_t n = shape_tiles(shape, M, N), full = n / kCus, rem = n % kCus;
    const double with_rem = step_us(t, shape, full + (rem ? 1 : 0)), without = step_us(t, shape, full);
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && (rem * s > kCus || rem == 0 || steps < 4 * s)) break;
      // the CUs work on full + 1 tiles until the split ones end, then on the others
      const double us = (double)steps * (with_rem / s + without * (1.0 - 1.0 / s)) +
                        (s > 1 ? partials_us((double)s * rem * kShapeTile[shape] * kShapeTile[shape]) : 0.0);
      if (us < 0.97 * best_us) best_us = us, best = {shape, s > 1 ? n - rem : n, s};
    }
  }
  return best;
}

// row pitch that a 256-row tile's 32-bit byte offsets can hold
constexpr int64_t kMaxRowBytes = int64_t(1) << 22;

// ---- vocabulary cross entropy (cross_entropy.hip)
bool ce_grid_fits(int64_t T, int64_t V, int d, int32_t dt);
size_t ce_workspace_bytes(int64_t T, int64_t V, int d, int32_t dt);
size_t ce_grad_workspace_bytes(int64_t T, int64_t V, int d, int32_t dt);
int launch_cross_entropy(const void* H, int32_t dt, int64_t T, int d, int64_t ldh, const void* W, int64_t V, int64_t ldw,
                         const int64_t* targets, float* loss, float* lse, void* ws, hipStream_t st);
int launch_cross_entropy_grad(const void* H, int32_t dt, int64_t T, int d, int64_t ldh, const void* W, int64_t V,
                              int64_t ldw, const int64_t* targets, const float* lse, const float* dloss, void* dH,
                              int64_t lddh, void* dW, int64_t lddw, void* ws, hipStream_t st);
int launch_zero_rows(void* out, int32_t dt, int64_t rows, int d, int64_t ldo, hipStream_t st);

}  // namespace qamw
