// The attention cache in microscaled 4-bit floating point (mxfp4.hip states
// the format): keys and values of new tokens quantised into the slots of a
// paged cache, and read back.
//
// Layout: codes [2][pages][heads][page][16 ceil(d / 32)] and scales
// [2][pages][heads][page][cache_scale_bytes(d)], keys first.  A page of one
// head is one run of memory, as attention reads it.  Slot s is place s % page
// of page s / page.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "mx4_device.h"
#include "qamw.h"
#include "qamw_device.h"
#include "qamw_internal.h"

namespace qamw {

// A row is one head of one token: 4 nb lanes of 8 elements, a quad of lanes a
// block.  blockIdx.y is 0 for keys and 1 for values.
struct CacheRow {
  int64_t token;
  int head, u;                                     // u: which 8 elements
  int64_t row;                                     // in the cache; -1: no such slot
};
template <class F>
__device__ __forceinline__ void each_cache_row(const CacheShape& c, const int64_t* __restrict__ slots, int64_t T, F&& f) {
  const int lanes = 4 * c.nb, per_block = kBlockThreads / lanes, sub = threadIdx.x / lanes;
  if (sub >= per_block) return;                    // whole quads leave
  const int64_t rows = T * c.heads, slots_all = c.pages << c.page_shift;
  for (int64_t r = (int64_t)blockIdx.x * per_block + sub; r < rows; r += (int64_t)gridDim.x * per_block) {
    CacheRow at;
    at.token = r / c.heads;
    at.head = (int)(r - at.token * c.heads);
    at.u = (int)threadIdx.x - sub * lanes;
    const int64_t slot = slots[at.token], page = slot >> c.page_shift;
    at.row = slot >= 0 && slot < slots_all
                 ? ((((int64_t)blockIdx.y * c.pages + page) * c.heads + at.head) << c.page_shift) + (slot & ((1 << c.page_shift) - 1))
                 : -1;
    f(at);
  }
}

struct TwoRows {                                   // keys and values in memory, [token][head][d] by strides
  const void* p[2];
  int64_t token[2], head[2];
};

template <class In>
__global__ __launch_bounds__(kBlockThreads) void cache_write_kernel(TwoRows in, int64_t T, CacheShape c,
                                                                    const int64_t* __restrict__ slots,
                                                                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int kv = blockIdx.y;
  each_cache_row(c, slots, T, [&](const CacheRow& at) {
    if (at.row < 0) return;                        // the same for a whole quad
    float x[8];
    load8<In>((const typename In::T*)in.p[kv] + at.token * in.token[kv] + at.head * in.head[kv], 8 * at.u, c.d, x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    const uint32_t code = scale_code(quad_max(m));
    *reinterpret_cast<uint32_t*>(codes + at.row * (16 * c.nb) + 4 * at.u) = encode8(x, code);
    uint8_t* srow = scales + at.row * c.sb;
    if ((at.u & 3) == 0) {
      srow[at.u >> 2] = (uint8_t)code;
      if (at.u == 4 * c.nb - 4)
        for (int q = c.nb; q < c.sb; ++q) srow[q] = 0;
    }
  });
}

template <class Out>
__global__ __launch_bounds__(kBlockThreads) void cache_read_kernel(TwoRows out, int64_t T, CacheShape c,
                                                                   const int64_t* __restrict__ slots,
                                                                   const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales) {
  const int kv = blockIdx.y;
  if (!out.p[kv]) return;
  each_cache_row(c, slots, T, [&](const CacheRow& at) {
    float x[8] = {};
    if (at.row >= 0)
      decode8(*reinterpret_cast<const uint32_t*>(codes + at.row * (16 * c.nb) + 4 * at.u), scales[at.row * c.sb + (at.u >> 2)], x);
    store8<Out>((typename Out::T*)out.p[kv] + at.token * out.token[kv] + at.head * out.head[kv], 8 * at.u, c.d, x);
  });
}

// ===========================================================================
// launchers
// ===========================================================================
static dim3 cache_grid(const CacheShape& c, int64_t T) {
  const int per_block = kBlockThreads / (4 * c.nb);
  return dim3((unsigned)std::min<int64_t>(tiles_of(T * c.heads, per_block), 1 << 20), 2);
}

template <class Mem>
static int write_from(const TwoRows& in, int64_t T, const CacheShape& c, const int64_t* slots, uint8_t* codes, uint8_t* scales,
                      hipStream_t st) {
  hipLaunchKernelGGL((cache_write_kernel<Mem>), cache_grid(c, T), dim3(kBlockThreads), 0, st, in, T, c, slots, codes, scales);
  return check_launch("cache_write_kernel");
}
int launch_cache_write(const void* K, const void* V, int32_t dt, int64_t T, int64_t kt, int64_t kh, int64_t vt, int64_t vh,
                       const CacheShape& c, const int64_t* slots, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const TwoRows in = {{K, V}, {kt, vt}, {kh, vh}};
  if (dt == QAMW_F32) return write_from<MemF32>(in, T, c, slots, codes, scales, st);
  if (dt == QAMW_F16) return write_from<MemF16>(in, T, c, slots, codes, scales, st);
  return write_from<MemBf16>(in, T, c, slots, codes, scales, st);
}

template <class Mem>
static int read_to(const TwoRows& out, int64_t T, const CacheShape& c, const int64_t* slots, const uint8_t* codes,
                   const uint8_t* scales, hipStream_t st) {
  hipLaunchKernelGGL((cache_read_kernel<Mem>), cache_grid(c, T), dim3(kBlockThreads), 0, st, out, T, c, slots, codes, scales);
  return check_launch("cache_read_kernel");
}
int launch_cache_read(void* K, void* V, int32_t dt, int64_t T, int64_t kt, int64_t kh, int64_t vt, int64_t vh,
                      const CacheShape& c, const int64_t* slots, const uint8_t* codes, const uint8_t* scales, hipStream_t st) {
  const TwoRows out = {{K, V}, {kt, vt}, {kh, vh}};
  if (dt == QAMW_F32) return read_to<MemF32>(out, T, c, slots, codes, scales, st);
  if (dt == QAMW_F16) return read_to<MemF16>(out, T, c, slots, codes, scales, st);
  return read_to<MemBf16>(out, T, c, slots, codes, scales, st);
}

}  // namespace qamw
