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
// block.  blockIdx.y is 0 for keys and 1 for values.  A lane takes kRows rows,
// a workgroup's width apart: slots, then elements, then results of all of them.
struct TwoRows {                                   // keys and values in memory, [token][head][d] by strides
  const void* p[2];
  int64_t token[2], head[2];
};
template <int kRows>
struct CacheRows {
  int64_t at[kRows];                               // row in the cache; -1: no such slot
  int64_t memory[kRows];                           // first element in memory
  bool in[kRows];
  int u;                                           // which 8 elements
  // false for lanes without work (whole quads)
  __device__ __forceinline__ bool find(const CacheShape& c, const int64_t* __restrict__ slots, uint32_t rows, const TwoRows& mem,
                                       uint32_t r0) {
    const int lanes = 4 * c.nb, per_block = kBlockThreads / lanes, sub = threadIdx.x / lanes, kv = blockIdx.y;
    u = (int)threadIdx.x - sub * lanes;
    if (sub >= per_block) return false;
    int64_t slot[kRows];
    uint32_t head[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t r = r0 + sub + i * per_block;
      in[i] = r < rows;
      const uint32_t token = (in[i] ? r : 0) / (uint32_t)c.heads;
      head[i] = (in[i] ? r : 0) - token * (uint32_t)c.heads;
      slot[i] = slots[token];
      memory[i] = token * mem.token[kv] + head[i] * mem.head[kv];
    }
    const int64_t all = c.pages << c.page_shift;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t block = (kv * c.pages + (slot[i] >> c.page_shift)) * c.heads + head[i];
      at[i] = slot[i] >= 0 && slot[i] < all ? (block << c.page_shift) + (slot[i] & ((1 << c.page_shift) - 1)) : -1;
    }
    return true;
  }
};

// Bound by memory where there is enough of it: 65536 tokens of 8 heads of 128
// read to bf16 take 76 us, 4.5 TB/s (99 us with one row a lane: a slot, then
// the codes, then the store wait for each other).
template <class In, int kRows>
__global__ __launch_bounds__(kBlockThreads) void cache_write_kernel(TwoRows in, uint32_t rows, CacheShape c,
                                                                    const int64_t* __restrict__ slots,
                                                                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint32_t per = kBlockThreads / (4 * c.nb) * kRows;
  for (uint32_t r0 = blockIdx.x * per; r0 < rows; r0 += gridDim.x * per) {
    CacheRows<kRows> row;
    if (!row.find(c, slots, rows, in, r0)) return;
    float x[kRows][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) load8<In>((const typename In::T*)in.p[blockIdx.y] + row.memory[i], 8 * row.u, c.d, x[i]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (!row.in[i] || row.at[i] < 0) continue;   // the same for a whole quad
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[i][e]) & 0x7fffffffu);
      const uint32_t code = scale_code(quad_max(m));
      *reinterpret_cast<uint32_t*>(codes + row.at[i] * (16 * c.nb) + 4 * row.u) = encode8(x[i], code);
      uint8_t* srow = scales + row.at[i] * c.sb;
      if ((row.u & 3) == 0) {
        srow[row.u >> 2] = (uint8_t)code;
        if (row.u == 4 * c.nb - 4)
          for (int q = c.nb; q < c.sb; ++q) srow[q] = 0;
      }
    }
  }
}

template <class Out, int kRows>
__global__ __launch_bounds__(kBlockThreads) void cache_read_kernel(TwoRows out, uint32_t rows, CacheShape c,
                                                                   const int64_t* __restrict__ slots,
                                                                   const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales) {
  if (!out.p[blockIdx.y]) return;
  const uint32_t per = kBlockThreads / (4 * c.nb) * kRows;
  for (uint32_t r0 = blockIdx.x * per; r0 < rows; r0 += gridDim.x * per) {
    CacheRows<kRows> row;
    if (!row.find(c, slots, rows, out, r0)) return;
    uint32_t code[kRows], scale[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      code[i] = scale[i] = 0;
      if (row.at[i] < 0) continue;
      code[i] = *reinterpret_cast<const uint32_t*>(codes + row.at[i] * (16 * c.nb) + 4 * row.u);
      scale[i] = scales[row.at[i] * c.sb + (row.u >> 2)];
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (!row.in[i]) continue;
      float x[8];
      decode8(code[i], scale[i], x);
      store8<Out>((typename Out::T*)out.p[blockIdx.y] + row.memory[i], 8 * row.u, c.d, x);
    }
  }
}

// ===========================================================================
// launchers
// ===========================================================================
// 4 rows a lane where that still gives every CU 4 workgroups, keys and values together
static bool four_rows(const CacheShape& c, int64_t T) { return T * c.heads >= 8ll * kCus * (kBlockThreads / (4 * c.nb)); }
static dim3 cache_grid(const CacheShape& c, int64_t T) {
  const int64_t per_block = kBlockThreads / (4 * c.nb) * (four_rows(c, T) ? 4 : 1);
  return dim3((unsigned)std::min<int64_t>(tiles_of(T * c.heads, per_block), 1 << 20), 2);
}

template <class Mem>
static int write_from(const TwoRows& in, int64_t T, const CacheShape& c, const int64_t* slots, uint8_t* codes, uint8_t* scales,
                      hipStream_t st) {
  auto kernel = four_rows(c, T) ? cache_write_kernel<Mem, 4> : cache_write_kernel<Mem, 1>;
  hipLaunchKernelGGL(kernel, cache_grid(c, T), dim3(kBlockThreads), 0, st, in, (uint32_t)(T * c.heads), c, slots, codes, scales);
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
  auto kernel = four_rows(c, T) ? cache_read_kernel<Mem, 4> : cache_read_kernel<Mem, 1>;
  hipLaunchKernelGGL(kernel, cache_grid(c, T), dim3(kBlockThreads), 0, st, out, (uint32_t)(T * c.heads), c, slots, codes, scales);
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
