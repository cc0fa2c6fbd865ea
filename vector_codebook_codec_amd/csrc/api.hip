// C ABI of libqamw.so (declared in include/qamw.h): argument validation on
// the host, then the stage launchers of calibrate.hip, encode.hip, plan.hip
// and decode.hip on the caller's stream.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdarg.h>
#include <stdint.h>

#include <algorithm>
#include <cstdio>
#include <mutex>
#include <string>

#include "qamw.h"
#include "qamw_internal.h"

namespace qamw {

thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(QAMW_EHIP, "%s: %s", what, hipGetErrorString(e));
  return QAMW_OK;
}

int log2_exact(int64_t v) {
  if (v <= 0 || (v & (v - 1))) return -1;
  int l = 0;
  while ((int64_t(1) << l) < v) ++l;
  return l;
}

int check_matrix(int64_t N, int64_t d, int32_t block, int* L) {
  if (N <= 0 || d <= 0) return fail(QAMW_EINVAL, "N and d must be positive (N=%lld d=%lld)", (long long)N, (long long)d);
  // every wavefront index (rows x 1024-column windows) must fit in an int
  if (N > kMaxDim || d > kMaxDim || N * ((d + 1023) / 1024) > (int64_t(1) << 30))
    return fail(QAMW_EUNSUPPORTED, "matrix too large");
  *L = log2_exact(block);
  if (*L < 1 || *L > 10) return fail(QAMW_EUNSUPPORTED, "block must be a power of two in [2, 1024] (got %d)", block);
  if (d % block) return fail(QAMW_EINVAL, "d=%lld is not a multiple of block=%d", (long long)d, block);
  // a lane owns 16 columns: with blocks under 16 the row must still be whole 16-column chunks
  if (d % 16) return fail(QAMW_EUNSUPPORTED, "d=%lld is not a multiple of 16", (long long)d);
  return QAMW_OK;
}

int check_weights(const void* W, int32_t wdt, int64_t d, int64_t ldw) {
  if (!W) return fail(QAMW_EINVAL, "W is NULL");
  if (wdt != QAMW_F32 && wdt != QAMW_BF16) return fail(QAMW_EUNSUPPORTED, "weight dtype %d not supported", wdt);
  if (ldw < d) return fail(QAMW_EINVAL, "ldw=%lld < d=%lld", (long long)ldw, (long long)d);
  if (!aligned16(W) || !rows_aligned16(ldw, wdt))
    return fail(QAMW_EINVAL, "W must be 16-byte aligned with 16-byte aligned rows");
  return QAMW_OK;
}

int check_codebook(const float* cb, int32_t K) {
  if (!cb) return fail(QAMW_EINVAL, "codebook is NULL");
  if (!aligned16(cb)) return fail(QAMW_EINVAL, "codebook must be 16-byte aligned");
  if (K < 2 || K > 4096) return fail(QAMW_EUNSUPPORTED, "K=%d outside [2, 4096]", K);
  return QAMW_OK;
}

// A search plan passed to an encode: NULL, or 256-byte aligned with at least
// plan_bytes(K) bytes (the kernels read that much of it).
int check_plan(const void* plan, size_t plan_size, int32_t K) {
  if (!plan) return QAMW_OK;
  if ((uintptr_t)plan & 255u) return fail(QAMW_EINVAL, "plan must be 256-byte aligned");
  if (plan_size < plan_bytes(K))
    return fail(QAMW_EWORKSPACE, "a plan for K=%d needs %zu bytes (got %zu)", (int)K, plan_bytes(K), plan_size);
  return QAMW_OK;
}

}  // namespace qamw

// ===========================================================================
// C ABI
// ===========================================================================
using namespace qamw;

extern "C" {

int32_t qamw_index_bits(int32_t K) {
  if (K < 2 || K > 4096) return -1;
  int32_t b = 0;
  while ((1 << b) < K) ++b;
  return b;
}

int64_t qamw_packed_row_words(int64_t d, int32_t K) {
  const int32_t B = qamw_index_bits(K);
  if (B < 0 || d <= 0 || (d & 1) || d > kMaxDim) return -1;
  const int64_t words = ((d / 2) * B + 31) / 32;
  return (words + 3) / 4 * 4;
}

size_t qamw_calibrate_workspace_bytes(int64_t N, int64_t d, int32_t block) {
  (void)block;
  if (N <= 0 || d <= 0 || N > kMaxDim || d > kMaxDim) return 0;
  return round_up((size_t)N * sizeof(double), 256) + round_up((size_t)d * sizeof(float), 256) +
         calib_tiles(N, d) * (size_t)(d / 2) * sizeof(float);
}

size_t qamw_encode_workspace_bytes(int64_t N, int64_t d) {
  if (N <= 0 || N > kMaxDim || d <= 0 || d > kMaxDim) return 0;
  return round_up((size_t)N * sizeof(double), 256) + round_up((size_t)d * sizeof(float), 256) +
         round_up((size_t)(d / 2) * sizeof(float), 256);
}

const char* qamw_status_string(int32_t status) {
  switch (status) {
    case QAMW_OK: return "ok";
    case QAMW_EINVAL: return "invalid argument";
    case QAMW_EUNSUPPORTED: return "unsupported argument";
    case QAMW_EHIP: return "HIP runtime error";
    case QAMW_EWORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
  }
}

const char* qamw_last_error(void) { return g_last_error.c_str(); }

const char* qamw_version(void) { return "qamw 0.1 gfx950"; }

int32_t qamw_calibrate(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, const float* chan_rms,
                       float alpha, int32_t block, uint64_t sign_seed, float* s_out, float* sigma_out,
                       void* workspace, size_t workspace_bytes, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if (!chan_rms || !s_out || !sigma_out) return fail(QAMW_EINVAL, "chan_rms, s_out and sigma_out must be non-NULL");
  if (!aligned16(s_out) || !aligned16(sigma_out)) return fail(QAMW_EINVAL, "s_out and sigma_out must be 16-byte aligned");
  if (!isfinite(alpha)) return fail(QAMW_EINVAL, "alpha must be finite");
  const size_t need = qamw_calibrate_workspace_bytes(N, d, block);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "calibrate needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  hipStream_t st = (hipStream_t)stream;
  double* rho = (double*)workspace;
  float* fcol = (float*)((char*)workspace + round_up((size_t)N * sizeof(double), 256));
  float* partial = (float*)((char*)fcol + round_up((size_t)d * sizeof(float), 256));
  const int n = (int)N, dd = (int)d;
  if ((rc = launch_scale(chan_rms, alpha, sign_seed, dd, s_out, fcol, st))) return rc;
  if ((rc = launch_norm_amplitude(L, W, wdtype, n, dd, ldw, s_out, fcol, rho, nullptr, partial, st))) return rc;
  return launch_sigma(partial, (int)calib_tiles(N, d), dd / 2, n, sigma_out, nullptr, st);
}

size_t qamw_plan_bytes(int32_t K) {
  if (K < 2 || K > 4096) return 0;
  return plan_bytes(K);
}

int32_t qamw_build_plan(const float* codebook, int32_t K, void* plan, size_t plan_size, void* stream) {
  int rc = check_codebook(codebook, K);
  if (rc) return rc;
  if (!plan || ((uintptr_t)plan & 255u)) return fail(QAMW_EINVAL, "plan must be non-NULL and 256-byte aligned");
  if (plan_size < plan_bytes(K))
    return fail(QAMW_EWORKSPACE, "plan needs %zu bytes (got %zu)", plan_bytes(K), plan_size);
  return launch_build_plan(codebook, K, plan, (hipStream_t)stream);
}

struct EncodeWorkspace {
  double* rho;    // [N] fp64 row factors 1 / (sqrt(b) rho_n) (0 for rho_n = 0)
  float* f;       // [d] eps_j s_j
  float* isig;    // [d/2] 1 / sigma_k
};

static EncodeWorkspace encode_workspace(void* workspace, int64_t N, int64_t d) {
  char* ws = (char*)workspace;
  EncodeWorkspace e;
  e.rho = (double*)ws;
  ws += round_up((size_t)N * sizeof(double), 256);
  e.f = (float*)ws;
  ws += round_up((size_t)d * sizeof(float), 256);
  e.isig = (float*)ws;
  return e;
}

static int check_encode_workspace(const void* workspace, size_t workspace_bytes, int64_t N, int64_t d) {
  const size_t need = qamw_encode_workspace_bytes(N, d);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "encode needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  return QAMW_OK;
}

int32_t qamw_encode_prepare(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, const float* s,
                            const float* sigma, int32_t block, uint64_t sign_seed, uint16_t* rownorm_f16,
                            void* workspace, size_t workspace_bytes, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if (!s || !sigma || !rownorm_f16) return fail(QAMW_EINVAL, "s, sigma and rownorm_f16 must be non-NULL");
  if (!aligned16(s) || !aligned16(sigma)) return fail(QAMW_EINVAL, "s and sigma must be 16-byte aligned");
  if ((rc = check_encode_workspace(workspace, workspace_bytes, N, d))) return rc;
  hipStream_t st = (hipStream_t)stream;
  const EncodeWorkspace e = encode_workspace(workspace, N, d);
  return launch_encode_prepare(L, W, wdtype, (int)N, (int)d, ldw, s, sigma, sign_seed, e.rho, rownorm_f16, e.f, e.isig,
                               st);
}

int32_t qamw_encode_indices(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, int32_t block,
                            const float* codebook, int32_t K, const void* plan, size_t plan_size, uint32_t* packed,
                            const void* workspace, size_t workspace_bytes, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if ((rc = check_codebook(codebook, K))) return rc;
  if (!packed) return fail(QAMW_EINVAL, "packed must be non-NULL");
  if (!aligned16(packed)) return fail(QAMW_EINVAL, "packed must be 16-byte aligned");
  if ((rc = check_plan(plan, plan_size, K))) return rc;
  if ((rc = check_encode_workspace(workspace, workspace_bytes, N, d))) return rc;
  const EncodeWorkspace e = encode_workspace(const_cast<void*>(workspace), N, d);
  return launch_encode(L, W, wdtype, (int)N, (int)d, ldw, e.f, e.isig, codebook, (int)K, qamw_index_bits(K),
                       (int)qamw_packed_row_words(d, K), e.rho, plan, packed, (hipStream_t)stream);
}

int32_t qamw_encode(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, const float* s,
                    const float* sigma, int32_t block, uint64_t sign_seed, const float* codebook, int32_t K,
                    const void* plan, size_t plan_size, uint32_t* packed, uint16_t* rownorm_f16, void* workspace,
                    size_t workspace_bytes, void* stream) {
  // validate everything before the first launch
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if ((rc = check_codebook(codebook, K))) return rc;
  if (!s || !sigma || !packed || !rownorm_f16) return fail(QAMW_EINVAL, "s, sigma, packed and rownorm_f16 must be non-NULL");
  if (!aligned16(s) || !aligned16(sigma) || !aligned16(packed))
    return fail(QAMW_EINVAL, "s, sigma and packed must be 16-byte aligned");
  if ((rc = check_plan(plan, plan_size, K))) return rc;
  if ((rc = check_encode_workspace(workspace, workspace_bytes, N, d))) return rc;
  if ((rc = qamw_encode_prepare(W, wdtype, N, d, ldw, s, sigma, block, sign_seed, rownorm_f16, workspace,
                                workspace_bytes, stream)))
    return rc;
  return qamw_encode_indices(W, wdtype, N, d, ldw, block, codebook, K, plan, plan_size, packed, workspace,
                             workspace_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// The no-allocation encode keeps qamw_encode's workspace (row norms, column
// factors, 1 / sigma) in this file-scope device array instead of a caller
// buffer.  Each GPU holds its own copy until the process ends; its device
// address is looked up once per device (hipGetSymbolAddress, with the device
// current) and every later call on that device uses that address.  All calls
// on one GPU share the array: calls that overlap on one GPU (different
// streams, or host threads) race and must be ordered by the caller.  Nothing
// in it has to start at zero: the encode writes every byte it reads.
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

int scratch_for_current_device(void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
    return fail(QAMW_EHIP, "cannot query the current device for the no-allocation scratch");
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p) return fail(QAMW_EHIP, "hipGetSymbolAddress(scratch): %s", hipGetErrorString(e));
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return QAMW_OK;
}
}  // namespace

extern "C" {

size_t qamw_encode_noalloc_scratch_bytes(void) { return kNoAllocScratchBytes; }

int32_t qamw_encode_noalloc(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, const float* s,
                            const float* sigma, int32_t block, uint64_t sign_seed, const float* codebook, int32_t K,
                            const void* plan, size_t plan_size, uint32_t* packed, uint16_t* rownorm_f16,
                            void* stream) {
  // the size limit first (host only), then everything qamw_encode checks
  const size_t need = qamw_encode_workspace_bytes(N, d);
  if (need > kNoAllocScratchBytes)
    return fail(QAMW_EUNSUPPORTED,
                "the no-allocation encode holds %zu bytes of workspace per GPU; N=%lld d=%lld needs %zu "
                "(use qamw_encode with a workspace)",
                kNoAllocScratchBytes, (long long)N, (long long)d, need);
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if ((rc = check_codebook(codebook, K))) return rc;
  if (!s || !sigma || !packed || !rownorm_f16) return fail(QAMW_EINVAL, "s, sigma, packed and rownorm_f16 must be non-NULL");
  if (!aligned16(s) || !aligned16(sigma) || !aligned16(packed))
    return fail(QAMW_EINVAL, "s, sigma and packed must be 16-byte aligned");
  if ((rc = check_plan(plan, plan_size, K))) return rc;
  void* ws = nullptr;
  if ((rc = scratch_for_current_device(&ws))) return rc;
  return qamw_encode(W, wdtype, N, d, ldw, s, sigma, block, sign_seed, codebook, K, plan, plan_size, packed,
                     rownorm_f16, ws, kNoAllocScratchBytes, stream);
}

size_t qamw_calibrate_encode_workspace_bytes(int64_t N, int64_t d) {
  const size_t e = qamw_encode_workspace_bytes(N, d);
  if (!e) return 0;
  return e + calib_tiles(N, d) * (size_t)(d / 2) * sizeof(float);
}

int32_t qamw_calibrate_prepare(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw,
                               const float* chan_rms, float alpha, int32_t block, uint64_t sign_seed, float* s_out,
                               float* sigma_out, uint16_t* rownorm_f16, void* workspace, size_t workspace_bytes,
                               void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if (!chan_rms || !s_out || !sigma_out || !rownorm_f16)
    return fail(QAMW_EINVAL, "chan_rms, s_out, sigma_out and rownorm_f16 must be non-NULL");
  if (!aligned16(s_out) || !aligned16(sigma_out)) return fail(QAMW_EINVAL, "s_out and sigma_out must be 16-byte aligned");
  if (!isfinite(alpha)) return fail(QAMW_EINVAL, "alpha must be finite");
  const size_t need = qamw_calibrate_encode_workspace_bytes(N, d);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "calibrate_prepare needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  hipStream_t st = (hipStream_t)stream;
  const EncodeWorkspace e = encode_workspace(workspace, N, d);
  float* partial = (float*)((char*)workspace + qamw_encode_workspace_bytes(N, d));
  const int n = (int)N, dd = (int)d;
  // the calibration pass leaves exactly what qamw_encode_prepare would compute:
  // column factors (scale_kernel), row norms with their fp16 bits
  // (norm_amplitude_kernel) and 1 / sigma (sigma_kernel)
  if ((rc = launch_scale(chan_rms, alpha, sign_seed, dd, s_out, e.f, st))) return rc;
  if ((rc = launch_norm_amplitude(L, W, wdtype, n, dd, ldw, s_out, e.f, e.rho, rownorm_f16, partial, st))) return rc;
  return launch_sigma(partial, (int)calib_tiles(N, d), dd / 2, n, sigma_out, e.isig, st);
}

int32_t qamw_calibrate_encode(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw,
                              const float* chan_rms, float alpha, int32_t block, uint64_t sign_seed,
                              const float* codebook, int32_t K, const void* plan, size_t plan_size, float* s_out,
                              float* sigma_out, uint32_t* packed, uint16_t* rownorm_f16, void* workspace,
                              size_t workspace_bytes, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if ((rc = check_codebook(codebook, K))) return rc;
  if (!chan_rms || !s_out || !sigma_out || !packed || !rownorm_f16)
    return fail(QAMW_EINVAL, "chan_rms, s_out, sigma_out, packed and rownorm_f16 must be non-NULL");
  if (!aligned16(s_out) || !aligned16(sigma_out) || !aligned16(packed))
    return fail(QAMW_EINVAL, "s_out, sigma_out and packed must be 16-byte aligned");
  if (!isfinite(alpha)) return fail(QAMW_EINVAL, "alpha must be finite");
  if ((rc = check_plan(plan, plan_size, K))) return rc;
  const size_t need = qamw_calibrate_encode_workspace_bytes(N, d);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "calibrate_encode needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  if ((rc = qamw_calibrate_prepare(W, wdtype, N, d, ldw, chan_rms, alpha, block, sign_seed, s_out, sigma_out,
                                   rownorm_f16, workspace, workspace_bytes, stream)))
    return rc;
  const EncodeWorkspace e = encode_workspace(workspace, N, d);
  return launch_encode(L, W, wdtype, (int)N, (int)d, ldw, e.f, e.isig, codebook, (int)K, qamw_index_bits(K),
                       (int)qamw_packed_row_words(d, K), e.rho, plan, packed, (hipStream_t)stream);
}

size_t qamw_lloyd_workspace_bytes(int32_t K) {
  if (K < 2 || K > 4096) return 0;
  return round_up((size_t)3 * K * sizeof(unsigned long long), 256) + round_up((size_t)kLloydMaxParts * sizeof(double), 256) +
         round_up((size_t)2 * K * sizeof(float), 256);
}

int32_t qamw_lloyd_update(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, int32_t block,
                          const uint32_t* packed, const float* codebook, int32_t K, const void* enc_workspace,
                          size_t enc_workspace_bytes, float* codebook_out, double* distortion_out,
                          void* workspace, size_t workspace_bytes, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if ((rc = check_codebook(codebook, K))) return rc;
  if (!packed || !aligned16(packed)) return fail(QAMW_EINVAL, "packed must be non-NULL and 16-byte aligned");
  if (!codebook_out || !aligned16(codebook_out)) return fail(QAMW_EINVAL, "codebook_out must be non-NULL and 16-byte aligned");
  if (codebook_out == codebook) return fail(QAMW_EINVAL, "codebook_out must not be the input codebook");
  if (!distortion_out || ((uintptr_t)distortion_out & 7u)) return fail(QAMW_EINVAL, "distortion_out must be non-NULL and 8-byte aligned");
  if ((rc = check_encode_workspace(enc_workspace, enc_workspace_bytes, N, d))) return rc;
  const size_t need = qamw_lloyd_workspace_bytes(K);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "lloyd update needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  const EncodeWorkspace e = encode_workspace(const_cast<void*>(enc_workspace), N, d);
  unsigned long long* gacc = (unsigned long long*)workspace;
  double* partial = (double*)((char*)workspace + round_up((size_t)3 * K * sizeof(unsigned long long), 256));
  return launch_lloyd_update(L, W, wdtype, (int)N, (int)d, ldw, e.f, e.isig, e.rho, packed,
                             (int)qamw_packed_row_words(d, K), qamw_index_bits(K), codebook, (int)K, codebook_out,
                             distortion_out, gacc, partial, (hipStream_t)stream);
}

int32_t qamw_learn_codebook(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, int32_t block,
                            const void* enc_workspace, size_t enc_workspace_bytes, const float* codebook_init,
                            int32_t K, int32_t iters, float* codebook_out, double* distortion_out, void* plan,
                            size_t plan_size, uint32_t* packed, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if ((rc = check_codebook(codebook_init, K))) return rc;
  if (iters < 1) return fail(QAMW_EINVAL, "iters must be >= 1 (got %d)", (int)iters);
  if (!codebook_out || !aligned16(codebook_out) || codebook_out == codebook_init)
    return fail(QAMW_EINVAL, "codebook_out must be non-NULL, 16-byte aligned and not the initial codebook");
  if (!distortion_out || ((uintptr_t)distortion_out & 7u)) return fail(QAMW_EINVAL, "distortion_out must be non-NULL and 8-byte aligned");
  if (!packed || !aligned16(packed)) return fail(QAMW_EINVAL, "packed must be non-NULL and 16-byte aligned");
  if (!plan || ((uintptr_t)plan & 255u) || plan_size < plan_bytes(K))
    return fail(QAMW_EWORKSPACE, "plan must be 256-byte aligned with %zu bytes", plan_bytes(K));
  if ((rc = check_encode_workspace(enc_workspace, enc_workspace_bytes, N, d))) return rc;
  const size_t need = qamw_lloyd_workspace_bytes(K);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "learn_codebook needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  hipStream_t st = (hipStream_t)stream;
  const EncodeWorkspace e = encode_workspace(const_cast<void*>(enc_workspace), N, d);
  unsigned long long* gacc = (unsigned long long*)workspace;
  double* partial = (double*)((char*)workspace + round_up((size_t)3 * K * sizeof(unsigned long long), 256));
  float* spare = (float*)((char*)partial + round_up((size_t)kLloydMaxParts * sizeof(double), 256));
  const int B = qamw_index_bits(K), rw = (int)qamw_packed_row_words(d, K);
  // round t reads cur and writes dst; the last round writes codebook_out
  const float* cur = codebook_init;
  for (int t = 0; t < iters; ++t) {
    float* dst = ((iters - 1 - t) % 2 == 0) ? codebook_out : spare;
    if ((rc = launch_build_plan(cur, (int)K, plan, st))) return rc;
    if ((rc = launch_encode(L, W, wdtype, (int)N, (int)d, ldw, e.f, e.isig, cur, (int)K, B, rw, e.rho, plan, packed,
                            st)))
      return rc;
    if ((rc = launch_lloyd_update(L, W, wdtype, (int)N, (int)d, ldw, e.f, e.isig, e.rho, packed, rw, B, cur, (int)K,
                                  dst, distortion_out + t, gacc, partial, st)))
      return rc;
    cur = dst;
  }
  return QAMW_OK;
}

int32_t qamw_encode_polar(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, const float* s,
                          const float* sigma, int32_t block, uint64_t sign_seed, const float* levels, int32_t Ka,
                          const float* dirs, int32_t Kp, uint32_t* packed, uint16_t* rownorm_f16, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_weights(W, wdtype, d, ldw))) return rc;
  if (!levels || !dirs) return fail(QAMW_EINVAL, "levels and dirs must be non-NULL");
  if (Ka < 1 || Kp < 1 || (int64_t)Ka * Kp < 2 || (int64_t)Ka * Kp > 4096)
    return fail(QAMW_EUNSUPPORTED, "polar code needs Ka, Kp >= 1 and 2 <= Ka * Kp <= 4096 (got %d x %d)", (int)Ka,
                (int)Kp);
  if (!s || !sigma || !packed || !rownorm_f16) return fail(QAMW_EINVAL, "s, sigma, packed and rownorm_f16 must be non-NULL");
  if (!aligned16(s) || !aligned16(sigma) || !aligned16(packed))
    return fail(QAMW_EINVAL, "s, sigma and packed must be 16-byte aligned");
  if ((rc = check_encode_workspace(workspace, workspace_bytes, N, d))) return rc;
  if ((rc = qamw_encode_prepare(W, wdtype, N, d, ldw, s, sigma, block, sign_seed, rownorm_f16, workspace,
                                workspace_bytes, stream)))
    return rc;
  const int K = Ka * Kp;
  const EncodeWorkspace e = encode_workspace(workspace, N, d);
  return launch_encode_polar(L, W, wdtype, (int)N, (int)d, ldw, e.f, e.isig, levels, (int)Ka, dirs, (int)Kp,
                             qamw_index_bits(K), (int)qamw_packed_row_words(d, K), e.rho, packed,
                             (hipStream_t)stream);
}

size_t qamw_channel_rms_workspace_bytes(int64_t T, int64_t d) {
  if (T <= 0 || T > kMaxDim || d <= 0 || d > kMaxDim) return 0;
  return round_up((size_t)((T + kRmsRowsPerTile - 1) / kRmsRowsPerTile) * (size_t)d * sizeof(float), 256);
}

static size_t oe_partials_bytes(int64_t T, int64_t N) {
  // one per workgroup: row blocks rounded up to whole groups of 8 (one per XCD) x token blocks
  const int64_t nb = (N + kOutputErrorRows - 1) / kOutputErrorRows;
  return round_up((size_t)((nb + 7) / 8 * 8) * (size_t)((T + kOutputErrorTokens - 1) / kOutputErrorTokens) *
                      sizeof(double), 256);
}

size_t qamw_output_error_workspace_bytes(int64_t T, int64_t N, int64_t d) {
  if (T <= 0 || T > kMaxDim || N <= 0 || N > kMaxDim || d <= 0 || d > kMaxDim) return 0;
  return oe_partials_bytes(T, N) + round_up((size_t)N * (size_t)d * 2, 256) + round_up((size_t)T * (size_t)d * 2, 256);
}

static int check_rows16(const void* p, int32_t dt, int64_t d, int64_t ld, const char* name, bool allow_f16) {
  if (!p) return fail(QAMW_EINVAL, "%s is NULL", name);
  if (dt != QAMW_F32 && dt != QAMW_BF16 && !(allow_f16 && dt == QAMW_F16))
    return fail(QAMW_EUNSUPPORTED, "%s dtype %d not supported", name, dt);
  if (ld < d) return fail(QAMW_EINVAL, "%s: leading dimension %lld < d=%lld", name, (long long)ld, (long long)d);
  if (!aligned16(p) || !rows_aligned16(ld, dt))
    return fail(QAMW_EINVAL, "%s must be 16-byte aligned with 16-byte aligned rows", name);
  return QAMW_OK;
}

int32_t qamw_channel_rms(const void* X, int32_t xdtype, int64_t T, int64_t d, int64_t ldx, float* r_out,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (T <= 0 || d <= 0) return fail(QAMW_EINVAL, "T and d must be positive (T=%lld d=%lld)", (long long)T, (long long)d);
  if (T > kMaxDim || d > kMaxDim) return fail(QAMW_EUNSUPPORTED, "activations too large");
  if (d % 8) return fail(QAMW_EINVAL, "d=%lld is not a multiple of 8", (long long)d);
  int rc = check_rows16(X, xdtype, d, ldx, "X", false);
  if (rc) return rc;
  if (!r_out || !aligned16(r_out)) return fail(QAMW_EINVAL, "r_out must be non-NULL and 16-byte aligned");
  const size_t need = qamw_channel_rms_workspace_bytes(T, d);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "channel RMS needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  return launch_channel_rms(X, xdtype, (int)T, (int)d, ldx, r_out, (float*)workspace, (hipStream_t)stream);
}

int32_t qamw_output_error(const void* X, int32_t xdtype, int64_t T, int64_t d, int64_t ldx, const void* W,
                          int32_t wdtype, int64_t N, int64_t ldw, const void* W_hat, int32_t hdtype, int64_t ldh,
                          double* err_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (T <= 0 || d <= 0 || N <= 0)
    return fail(QAMW_EINVAL, "T, N and d must be positive (T=%lld N=%lld d=%lld)", (long long)T, (long long)N,
                (long long)d);
  if (T > kMaxDim || d > kMaxDim || N > kMaxDim) return fail(QAMW_EUNSUPPORTED, "operands too large");
  if (d % 16) return fail(QAMW_EINVAL, "d=%lld is not a multiple of 16", (long long)d);
  int rc;
  if ((rc = check_rows16(X, xdtype, d, ldx, "X", false))) return rc;
  if ((rc = check_rows16(W, wdtype, d, ldw, "W", false))) return rc;
  if ((rc = check_rows16(W_hat, hdtype, d, ldh, "W_hat", false))) return rc;
  if (!err_out || ((uintptr_t)err_out & 7u)) return fail(QAMW_EINVAL, "err_out must be non-NULL and 8-byte aligned");
  const size_t need = qamw_output_error_workspace_bytes(T, N, d);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "output error needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  char* ws = (char*)workspace;
  double* partial = (double*)ws;
  uint16_t* dWb = (uint16_t*)(ws + oe_partials_bytes(T, N));
  uint16_t* Xb = (uint16_t*)((char*)dWb + round_up((size_t)N * (size_t)d * 2, 256));
  return launch_output_error(X, xdtype, (int)T, (int)d, ldx, W, wdtype, (int)N, ldw, W_hat, hdtype, ldh, err_out,
                             partial, dWb, Xb, (hipStream_t)stream);
}

int32_t qamw_decode(const uint32_t* packed, const uint16_t* rownorm_f16, int64_t N, int64_t d, const float* s,
                    const float* sigma, int32_t block, uint64_t sign_seed, const float* codebook, int32_t K,
                    void* W_out, int32_t out_dtype, int64_t ldo, void* stream) {
  int L = 0;
  int rc = check_matrix(N, d, block, &L);
  if (rc) return rc;
  if ((rc = check_codebook(codebook, K))) return rc;
  if (!packed || !rownorm_f16 || !sigma || !W_out)
    return fail(QAMW_EINVAL, "packed, rownorm_f16, sigma and W_out must be non-NULL");
  if (out_dtype != QAMW_F32 && out_dtype != QAMW_BF16 && out_dtype != QAMW_F16)
    return fail(QAMW_EUNSUPPORTED, "output dtype %d not supported", out_dtype);
  if (ldo < d) return fail(QAMW_EINVAL, "ldo=%lld < d=%lld", (long long)ldo, (long long)d);
  if (!aligned16(packed) || !aligned16(W_out) || !rows_aligned16(ldo, out_dtype) || !aligned16(sigma) ||
      (s && !aligned16(s)))
    return fail(QAMW_EINVAL, "packed, s, sigma and W_out must be 16-byte aligned with 16-byte aligned rows");
  const int B = qamw_index_bits(K);
  const int row_words = (int)qamw_packed_row_words(d, K);
  return launch_decode(L, packed, rownorm_f16, (int)N, (int)d, s, sigma, sign_seed, codebook, (int)K, B, row_words,
                       W_out, out_dtype, ldo, (hipStream_t)stream);
}

int32_t qamw_rotate_activations(const void* X, int32_t xdtype, int64_t T, int64_t d, int64_t ldx, const float* s,
                                int32_t block, uint64_t sign_seed, uint16_t* Xr_bf16, int64_t ldr, void* stream) {
  int L = 0;
  int rc = check_matrix(T, d, block, &L);
  if (rc) return rc;
  if (!X) return fail(QAMW_EINVAL, "X is NULL");
  if (xdtype != QAMW_F32 && xdtype != QAMW_BF16) return fail(QAMW_EUNSUPPORTED, "activation dtype %d not supported", xdtype);
  if (ldx < d || ldr < d) return fail(QAMW_EINVAL, "ldx and ldr must be >= d");
  if (!Xr_bf16) return fail(QAMW_EINVAL, "Xr_bf16 is NULL");
  if (!aligned16(X) || !rows_aligned16(ldx, xdtype) || !aligned16(Xr_bf16) || ldr % 8 || (s && !aligned16(s)))
    return fail(QAMW_EINVAL, "X, Xr_bf16 and s must be 16-byte aligned with 16-byte aligned rows");
  return launch_rotate_act(L, X, xdtype, (int)T, (int)d, ldx, s, sign_seed, Xr_bf16, ldr, (hipStream_t)stream);
}

int32_t qamw_decode_matmul(const uint16_t* Xr_bf16, int64_t T, int64_t d, int64_t ldr, const uint32_t* packed,
                           const uint16_t* rownorm_f16, int64_t N, const float* sigma, const float* codebook,
                           int32_t K, void* Y, int32_t ydtype, int64_t ldy, void* stream) {
  if (T <= 0 || N <= 0 || d <= 0) return fail(QAMW_EINVAL, "T, N and d must be positive");
  if (T > kMaxDim || N > kMaxDim || d > kMaxDim) return fail(QAMW_EUNSUPPORTED, "matrix too large");
  if (d % 16) return fail(QAMW_EINVAL, "d=%lld is not a multiple of 16", (long long)d);
  int rc = check_codebook(codebook, K);
  if (rc) return rc;
  if (!Xr_bf16 || !packed || !rownorm_f16 || !sigma || !Y)
    return fail(QAMW_EINVAL, "Xr_bf16, packed, rownorm_f16, sigma and Y must be non-NULL");
  if (ydtype != QAMW_F32 && ydtype != QAMW_BF16) return fail(QAMW_EUNSUPPORTED, "output dtype %d not supported", ydtype);
  if (ldr < d || ldy < N) return fail(QAMW_EINVAL, "ldr must be >= d and ldy >= N");
  if (!aligned16(Xr_bf16) || ldr % 8 || !aligned16(packed) || !aligned16(sigma))
    return fail(QAMW_EINVAL, "Xr_bf16, packed and sigma must be 16-byte aligned, Xr rows too");
  const int B = qamw_index_bits(K);
  const int row_words = (int)qamw_packed_row_words(d, K);
  return launch_decode_matmul(Xr_bf16, (int)T, (int)d, ldr, packed, row_words, rownorm_f16, (int)N, sigma, codebook,
                              K, B, Y, ydtype, ldy, (hipStream_t)stream);
}

// ---------------- microscaled 4-bit floating point ----------------
constexpr int64_t kMx4MaxDim = int64_t(1) << 20;
constexpr int64_t kMaxRows = int64_t(1) << 31;

int64_t qamw_mxfp4_row_bytes(int64_t d) { return d >= 1 && d <= kMx4MaxDim ? mx4_blocks(d) * 16 : -1; }
int64_t qamw_mxfp4_scale_bytes(int64_t d) { return d >= 1 && d <= kMx4MaxDim ? mx4_scale_bytes(d) : -1; }

static int check_mx4(int64_t N, int64_t d, const void* codes, const void* scales) {
  if (N < 0 || d <= 0) return fail(QAMW_EINVAL, "sizes must not be negative and d positive (rows %lld, d=%lld)", (long long)N, (long long)d);
  if (N > kMaxRows || d > kMx4MaxDim) return fail(QAMW_EUNSUPPORTED, "matrix too large (rows %lld, d=%lld)", (long long)N, (long long)d);
  if (N && (!codes || !scales || !aligned16(codes) || !aligned16(scales)))
    return fail(QAMW_EINVAL, "codes and scales must be non-NULL and 16-byte aligned");
  return QAMW_OK;
}
// a matrix of any leading dimension, aligned to its elements
static int check_plain_rows(const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld, const char* name, bool f16) {
  if (dt != QAMW_F32 && dt != QAMW_BF16 && !(f16 && dt == QAMW_F16))
    return fail(QAMW_EUNSUPPORTED, "%s dtype %d not supported", name, dt);
  if (ld < cols) return fail(QAMW_EINVAL, "%s: leading dimension %lld < %lld", name, (long long)ld, (long long)cols);
  if (rows && (!p || (uintptr_t)p % (uintptr_t)elem_size(dt)))
    return fail(QAMW_EINVAL, "%s must be non-NULL and aligned to its elements", name);
  return QAMW_OK;
}

int32_t qamw_mxfp4_quantize(const void* W, int32_t wdtype, int64_t N, int64_t d, int64_t ldw, uint8_t* codes,
                            uint8_t* scales, void* values, int32_t vdtype, int64_t ldv, void* stream) {
  int rc = check_mx4(N, d, codes, scales);
  if (rc) return rc;
  if ((rc = check_plain_rows(W, wdtype, N, d, ldw, "W", true))) return rc;
  if (values && (rc = check_plain_rows(values, vdtype, N, d, ldv, "values", true))) return rc;
  if (N == 0) return QAMW_OK;
  return launch_mx4_quantize(W, wdtype, N, (int)d, ldw, codes, scales, values, values ? vdtype : QAMW_BF16, ldv,
                             (hipStream_t)stream);
}

int32_t qamw_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t d, void* W_out,
                              int32_t out_dtype, int64_t ldo, void* stream) {
  int rc = check_mx4(N, d, codes, scales);
  if (rc) return rc;
  if ((rc = check_plain_rows(W_out, out_dtype, N, d, ldo, "W_out", true))) return rc;
  if (N == 0) return QAMW_OK;
  return launch_mx4_dequantize(codes, scales, N, (int)d, W_out, out_dtype, ldo, (hipStream_t)stream);
}

size_t qamw_mxfp4_matmul_workspace_bytes(int64_t T, int64_t N, int64_t d) {
  if (T <= 0 || T > kMaxRows || N <= 0 || N > kMaxRows || d <= 0 || d > kMx4MaxDim) return 0;
  return mx4_matmul_workspace_bytes(T, N, d);
}

int32_t qamw_mxfp4_matmul(const void* X, int32_t xdtype, int64_t T, int64_t d, int64_t ldx, const uint8_t* codes,
                          const uint8_t* scales, int64_t N, void* Y, int32_t ydtype, int64_t ldy, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int rc = check_mx4(N, d, codes, scales);
  if (rc) return rc;
  if (T < 0) return fail(QAMW_EINVAL, "T must not be negative (T=%lld)", (long long)T);
  if (T > kMaxRows || (T && N && !mx4_grid_fits(T, N, d))) return fail(QAMW_EUNSUPPORTED, "product too large");
  if ((rc = check_plain_rows(X, xdtype, T, d, ldx, "X", true))) return rc;
  if ((rc = check_plain_rows(Y, ydtype, N ? T : 0, N, ldy, "Y", false))) return rc;
  if (T == 0 || N == 0) return QAMW_OK;
  const size_t need = qamw_mxfp4_matmul_workspace_bytes(T, N, d);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "the 4-bit product needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  return launch_mx4_matmul(X, xdtype, T, (int)d, ldx, codes, scales, N, Y, ydtype, ldy, workspace, nullptr, (hipStream_t)stream);
}

// the product's workspace first, then the adapters'
constexpr int64_t kMaxRank = 1024;
static bool adapter_sizes_fit(int64_t T, int64_t N, int64_t d, int64_t rank, int64_t n) {
  return n <= INT32_MAX && rank <= kMaxRank && (n <= 0 || T <= 0 || N <= 0 ||
                                                (adapter_grid_fits(T, N, rank) && N <= (int64_t(1) << 45) / (n * rank) &&
                                                 d <= (int64_t(1) << 45) / (n * rank)));
}
size_t qamw_mxfp4_adapter_matmul_workspace_bytes(int64_t T, int64_t N, int64_t d, int64_t rank, int32_t xdtype) {
  const size_t product = qamw_mxfp4_matmul_workspace_bytes(T, N, d);
  if (!product || rank <= 0 || rank > kMaxRank || (xdtype != QAMW_F32 && xdtype != QAMW_BF16)) return 0;
  return round_up(product, 256) + adapter_workspace_bytes(T, N, d, xdtype, rank);
}

int32_t qamw_mxfp4_adapter_matmul(const void* X, int32_t xdtype, int64_t T, int64_t d, int64_t ldx, const uint8_t* codes,
                                  const uint8_t* scales, int64_t N, const void* A, const void* B, int64_t adapters,
                                  int64_t rank, const int32_t* index, const float* factors, void* Y, int32_t ydtype,
                                  int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_mx4(N, d, codes, scales);
  if (rc) return rc;
  if (T < 0 || adapters < 0 || rank <= 0)
    return fail(QAMW_EINVAL, "T and adapters must not be negative and rank positive (T=%lld adapters=%lld rank=%lld)",
                (long long)T, (long long)adapters, (long long)rank);
  if (xdtype != QAMW_F32 && xdtype != QAMW_BF16) return fail(QAMW_EUNSUPPORTED, "X dtype %d not supported with adapters", xdtype);
  if (T > kMaxRows || (T && N && !mx4_grid_fits(T, N, d)) || !adapter_sizes_fit(T, N, d, rank, adapters))
    return fail(QAMW_EUNSUPPORTED, "product too large");
  if ((rc = check_plain_rows(X, xdtype, T, d, ldx, "X", false))) return rc;
  if ((rc = check_plain_rows(Y, ydtype, N ? T : 0, N, ldy, "Y", false))) return rc;
  if (T == 0 || N == 0) return QAMW_OK;
  if (adapters && (!A || !B || !aligned16(A) || !aligned16(B)))
    return fail(QAMW_EINVAL, "A and B must be non-NULL and 16-byte aligned");
  if (adapters && (!index || ((uintptr_t)index & 3u) || ((uintptr_t)factors & 3u)))
    return fail(QAMW_EINVAL, "index must be non-NULL, index and factors 4-byte aligned");
  const size_t need = qamw_mxfp4_adapter_matmul_workspace_bytes(T, N, d, rank, xdtype);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "the product with adapters needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  Adapters ad = {};
  ad.B = B, ad.index = index, ad.factors = factors, ad.n = (int)adapters, ad.rank = (int)rank;
  char* own = (char*)workspace + round_up(qamw_mxfp4_matmul_workspace_bytes(T, N, d), 256);
  if (adapters && (rc = launch_adapter_shrink(X, xdtype, T, N, d, ldx, A, own, &ad, (hipStream_t)stream))) return rc;
  return launch_mx4_matmul(X, xdtype, T, (int)d, ldx, codes, scales, N, Y, ydtype, ldy, workspace, adapters ? &ad : nullptr,
                           (hipStream_t)stream);
}

// ---------------- attention cache in 4 bits ----------------
constexpr int64_t kCacheMaxBytes = int64_t(1) << 45;
constexpr int64_t kCacheMaxTokens = int64_t(1) << 30;      // of a sequence, and query rows of a call

int64_t qamw_mxfp4_cache_row_bytes(int64_t d) { return d >= 1 && d <= kCacheMaxHeadDim ? mx4_blocks(d) * 16 : -1; }
int64_t qamw_mxfp4_cache_scale_bytes(int64_t d) { return d >= 1 && d <= kCacheMaxHeadDim ? cache_scale_bytes(d) : -1; }

static int check_cache(const void* codes, const void* scales, int64_t pages, int64_t heads, int64_t page, int64_t d,
                       CacheShape* c) {
  if (pages < 0 || heads <= 0 || d <= 0)
    return fail(QAMW_EINVAL, "heads and d must be positive and pages not negative (pages=%lld heads=%lld d=%lld)",
                (long long)pages, (long long)heads, (long long)d);
  const int shift = log2_exact(page);
  if (shift < 0 || page < kCacheMinPage || page > kCacheMaxPage)
    return fail(QAMW_EUNSUPPORTED, "a page must hold a power of two in [16, 65536] of tokens (got %lld)", (long long)page);
  if (d > kCacheMaxHeadDim) return fail(QAMW_EUNSUPPORTED, "head dimension %lld above 256", (long long)d);
  // a page of all heads is stepped over by 32 bits
  if (heads > 65536 || heads * page > (int64_t(1) << 31) / (mx4_blocks(d) * 16) || pages > kCacheMaxBytes / (heads * page * mx4_blocks(d) * 16) || pages > INT32_MAX)
    return fail(QAMW_EUNSUPPORTED, "cache too large");
  if (pages && (!codes || !scales || !aligned16(codes) || !aligned16(scales)))
    return fail(QAMW_EINVAL, "codes and scales must be non-NULL and 16-byte aligned");
  *c = {pages, (int)heads, shift, (int)d, (int)mx4_blocks(d), cache_scale_bytes(d)};
  return QAMW_OK;
}
// rows [T][heads][d] of any strides (unit stride along d), aligned to their elements; outputs may not overlap themselves
static int check_head_rows(const void* p, int32_t dt, int64_t T, int64_t heads, int64_t d, int64_t token, int64_t head,
                           const char* name, bool written) {
  if (dt != QAMW_F32 && dt != QAMW_BF16 && dt != QAMW_F16) return fail(QAMW_EUNSUPPORTED, "%s dtype %d not supported", name, dt);
  if (token < 0 || head < 0) return fail(QAMW_EINVAL, "%s: strides must not be negative", name);
  if (!T) return QAMW_OK;
  if (!p || (uintptr_t)p % (uintptr_t)elem_size(dt))
    return fail(QAMW_EINVAL, "%s must be non-NULL and aligned to its elements", name);
  if (token > kCacheMaxBytes || head > kCacheMaxBytes) return fail(QAMW_EUNSUPPORTED, "%s: strides too large", name);
  if (written) {
    // one stride steps over whole rows, the other over everything that the first spans
    const int64_t tokens = T - 1, others = heads - 1;
    const bool apart_h = heads == 1 || head >= d, apart_t = T == 1 || token >= d;
    const bool heads_in = T == 1 || heads == 1 || others <= (token - d) / (head ? head : 1);
    const bool tokens_in = T == 1 || heads == 1 || tokens <= (head - d) / (token ? token : 1);
    if (!apart_h || !apart_t || !(heads_in || tokens_in)) return fail(QAMW_EINVAL, "%s: rows overlap", name);
  }
  return QAMW_OK;
}
static int check_slots(const int64_t* slots, int64_t T, int64_t heads) {
  if (T < 0) return fail(QAMW_EINVAL, "T must not be negative (T=%lld)", (long long)T);
  if (T > kMaxRows / 2 / heads) return fail(QAMW_EUNSUPPORTED, "too many tokens (T=%lld)", (long long)T);
  if (T && (!slots || ((uintptr_t)slots & 7u))) return fail(QAMW_EINVAL, "slots must be non-NULL and 8-byte aligned");
  return QAMW_OK;
}

int32_t qamw_mxfp4_cache_write(const void* K, const void* V, int32_t dtype, int64_t T, int64_t heads, int64_t d,
                               int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, const int64_t* slots,
                               uint8_t* codes, uint8_t* scales, int64_t pages, int64_t page, void* stream) {
  CacheShape c;
  int rc = check_cache(codes, scales, pages, heads, page, d, &c);
  if (rc || (rc = check_slots(slots, T, heads)) || (rc = check_head_rows(K, dtype, T, heads, d, k_token, k_head, "K", false)) ||
      (rc = check_head_rows(V, dtype, T, heads, d, v_token, v_head, "V", false)))
    return rc;
  if (T == 0 || pages == 0) return QAMW_OK;
  return launch_cache_write(K, V, dtype, T, k_token, k_head, v_token, v_head, c, slots, codes, scales, (hipStream_t)stream);
}

int32_t qamw_mxfp4_cache_read(const uint8_t* codes, const uint8_t* scales, int64_t pages, int64_t page, int64_t heads, int64_t d,
                              const int64_t* slots, int64_t T, void* K, void* V, int32_t dtype, int64_t k_token,
                              int64_t k_head, int64_t v_token, int64_t v_head, void* stream) {
  CacheShape c;
  int rc = check_cache(codes, scales, pages, heads, page, d, &c);
  if (rc || (rc = check_slots(slots, T, heads)) ||
      (rc = check_head_rows(K, dtype, K ? T : 0, heads, d, k_token, k_head, "K", true)) ||
      (rc = check_head_rows(V, dtype, V ? T : 0, heads, d, v_token, v_head, "V", true)))
    return rc;
  if (T == 0 || (!K && !V)) return QAMW_OK;
  return launch_cache_read(K, V, dtype, T, k_token, k_head, v_token, v_head, c, slots, codes, scales, (hipStream_t)stream);
}

// sizes that a call's launches and 32-bit row indices can hold
static bool attention_sizes_fit(int64_t T, int64_t sequences, int64_t max_queries, int64_t heads, int64_t q_heads, int64_t tokens) {
  return T <= kCacheMaxTokens && heads <= 65536 && q_heads <= 65536 && sequences <= (int64_t(1) << 24) / heads &&
         T * (q_heads / heads) <= kCacheMaxTokens && max_queries >= 1 && tokens <= kCacheMaxTokens;
}
static AttentionPlan plan_of(int64_t T, int64_t sequences, int64_t max_queries, int64_t heads, int64_t q_heads, int64_t d,
                             int64_t tokens, int32_t qdt, int32_t odt) {
  return attention_plan(T, sequences, std::min(max_queries, T), heads, q_heads / heads, d, tokens, qdt, odt);
}
static bool attention_grid_fits(const AttentionPlan& p, int64_t T, int64_t q_heads) {
  return grid_holds(p.groups, kBlockThreads) && (p.splits == 1 || grid_holds(T * q_heads / 4 + 1, kBlockThreads));
}
size_t qamw_mxfp4_cache_attention_workspace_bytes(int64_t T, int64_t sequences, int64_t max_queries, int64_t heads,
                                                  int64_t q_heads, int64_t d, int64_t tokens, int32_t qdtype, int32_t odtype) {
  if (T <= 0 || sequences <= 0 || heads <= 0 || q_heads <= 0 || q_heads % heads || d <= 0 || d > kCacheMaxHeadDim || tokens < 0 ||
      !elem_size(qdtype) || !elem_size(odtype) || !attention_sizes_fit(T, sequences, max_queries, heads, q_heads, tokens))
    return 0;
  return plan_of(T, sequences, max_queries, heads, q_heads, d, tokens, qdtype, odtype).bytes;
}

int32_t qamw_mxfp4_cache_attention(const void* Q, int32_t qdtype, int64_t T, int64_t q_heads, int64_t d, int64_t q_token,
                                   int64_t q_head, const int32_t* starts, int64_t sequences, int64_t max_queries,
                                   const uint8_t* codes, const uint8_t* scales, int64_t pages, int64_t page, int64_t heads,
                                   const int32_t* table, int64_t table_cols, int64_t table_pitch, const int32_t* lengths,
                                   float scale, int32_t causal, int64_t window, void* out, int32_t odtype, int64_t o_token,
                                   int64_t o_head, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  AttentionArgs a;
  int rc = check_cache(codes, scales, pages, heads, page, d, &a.c);
  if (rc) return rc;
  if (T < 0 || sequences < 0 || q_heads <= 0 || q_heads % heads)
    return fail(QAMW_EINVAL, "sizes must not be negative and q_heads a multiple of heads (T=%lld sequences=%lld q_heads=%lld heads=%lld)",
                (long long)T, (long long)sequences, (long long)q_heads, (long long)heads);
  if (max_queries < 1 || (!starts && (max_queries != 1 || sequences != T)))
    return fail(QAMW_EINVAL, "max_queries must be positive; without starts there is one query a sequence");
  if (table_cols < 0 || table_pitch < table_cols) return fail(QAMW_EINVAL, "table_pitch must be >= table_cols >= 0");
  if (table_cols > kCacheMaxTokens / page || table_pitch > kCacheMaxBytes ||
      !attention_sizes_fit(T, sequences, max_queries, heads, q_heads, table_cols * page))
    return fail(QAMW_EUNSUPPORTED, "attention too large");
  if (!(scale > 0.0f) || isinf(scale)) return fail(QAMW_EINVAL, "scale must be positive and finite");
  if (window < 0) return fail(QAMW_EINVAL, "window must not be negative (0: none)");
  if ((rc = check_head_rows(Q, qdtype, T, q_heads, d, q_token, q_head, "Q", false)) ||
      (rc = check_head_rows(out, odtype, T, q_heads, d, o_token, o_head, "out", true)))
    return rc;
  if (T == 0 || sequences == 0) return QAMW_OK;
  if (!lengths || ((uintptr_t)lengths & 3u) || ((uintptr_t)starts & 3u) || (table_cols && !table) || ((uintptr_t)table & 3u))
    return fail(QAMW_EINVAL, "starts, lengths and table must be 4-byte aligned, lengths and table non-NULL");
  if ((uintptr_t)lse & 3u) return fail(QAMW_EINVAL, "lse must be 4-byte aligned");
  const int64_t tokens = table_cols * page;
  const AttentionPlan p = plan_of(T, sequences, max_queries, heads, q_heads, d, tokens, qdtype, odtype);
  if (!attention_grid_fits(p, T, q_heads)) return fail(QAMW_EUNSUPPORTED, "attention too large");
  if (p.bytes && (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 255u)))
    return fail(QAMW_EWORKSPACE, "the attention needs %zu bytes of 256-byte aligned workspace (got %zu)", p.bytes, workspace_bytes);
  a.codes = codes, a.scales = scales;
  a.Q = Q, a.qdt = qdtype, a.q_token = q_token, a.q_head = q_head;
  a.out = out, a.odt = odtype, a.o_token = o_token, a.o_head = o_head;
  a.lse = lse;
  a.starts = starts, a.lengths = lengths, a.table = table, a.table_pitch = table_pitch, a.cols = (int)table_cols;
  a.T = T;
  a.sequences = (int)sequences, a.group = (int)(q_heads / heads);
  a.most = (int)std::min(max_queries, T);
  a.scale = scale, a.causal = causal != 0;
  a.window = window >= kCacheMaxTokens ? 0 : (int)window;    // no narrower than any sequence
  return launch_cache_attention(a, p, workspace, (hipStream_t)stream);
}

// ---------------- vocabulary cross entropy ----------------
// sizes that the kernels' 32-bit offsets inside a tile and their grids can hold
static bool ce_sizes_fit(int64_t T, int64_t V, int64_t d, int32_t dtype) {
  const int64_t row = kMaxRowBytes / elem_size(dtype);      // compared before anything is multiplied: sizes may be of any value
  return V <= kMaxDim && d < row && T < row && (T <= 0 || ce_grid_fits(T, V, (int)d, dtype));
}
static int check_ce(const void* H, int32_t dtype, int64_t T, int64_t d, int64_t ldh, const void* W, int64_t V, int64_t ldw,
                    const int64_t* targets) {
  if (T < 0 || V <= 0 || d <= 0)
    return fail(QAMW_EINVAL, "V and d must be positive and T not negative (T=%lld V=%lld d=%lld)", (long long)T,
                (long long)V, (long long)d);
  if (dtype != QAMW_F32 && dtype != QAMW_BF16) return fail(QAMW_EUNSUPPORTED, "dtype %d not supported", dtype);
  if (d % 8) return fail(QAMW_EINVAL, "d=%lld is not a multiple of 8", (long long)d);
  if (!ce_sizes_fit(T, V, d, dtype)) return fail(QAMW_EUNSUPPORTED, "operands too large");
  int rc;
  if (T && (rc = check_rows16(H, dtype, d, ldh, "H", false))) return rc;
  if ((rc = check_rows16(W, dtype, d, ldw, "W", false))) return rc;
  const int64_t row = kMaxRowBytes / elem_size(dtype);
  if (ldh > row || ldw > row)
    return fail(QAMW_EUNSUPPORTED, "leading dimension too large");
  if (T && (!targets || ((uintptr_t)targets & 7u))) return fail(QAMW_EINVAL, "targets must be non-NULL and 8-byte aligned");
  return QAMW_OK;
}
static bool aligned4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }

size_t qamw_cross_entropy_workspace_bytes(int64_t T, int64_t V, int64_t d, int32_t dtype) {
  if (T <= 0 || V <= 0 || d <= 0 || (dtype != QAMW_F32 && dtype != QAMW_BF16) || !ce_sizes_fit(T, V, d, dtype)) return 0;
  return ce_workspace_bytes(T, V, (int)d, dtype);
}
size_t qamw_cross_entropy_grad_workspace_bytes(int64_t T, int64_t V, int64_t d, int32_t dtype) {
  if (T <= 0 || V <= 0 || d <= 0 || (dtype != QAMW_F32 && dtype != QAMW_BF16) || !ce_sizes_fit(T, V, d, dtype)) return 0;
  return ce_grad_workspace_bytes(T, V, (int)d, dtype);
}

int32_t qamw_cross_entropy(const void* H, int32_t dtype, int64_t T, int64_t d, int64_t ldh, const void* W, int64_t V,
                           int64_t ldw, const int64_t* targets, float* loss, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int rc = check_ce(H, dtype, T, d, ldh, W, V, ldw, targets);
  if (rc) return rc;
  if (T == 0) return QAMW_OK;
  if (!aligned4(loss) || !aligned4(lse)) return fail(QAMW_EINVAL, "loss and lse must be non-NULL and 4-byte aligned");
  const size_t need = qamw_cross_entropy_workspace_bytes(T, V, d, dtype);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "the cross entropy needs %zu bytes of 256-byte aligned workspace (got %zu)", need,
                workspace_bytes);
  return launch_cross_entropy(H, dtype, T, (int)d, ldh, W, V, ldw, targets, loss, lse, workspace, (hipStream_t)stream);
}

int32_t qamw_cross_entropy_grad(const void* H, int32_t dtype, int64_t T, int64_t d, int64_t ldh, const void* W,
                                int64_t V, int64_t ldw, const int64_t* targets, const float* lse, const float* dloss,
                                void* dH, int64_t lddh, void* dW, int64_t lddw, void* workspace,
                                size_t workspace_bytes, void* stream) {
  int rc = check_ce(H, dtype, T, d, ldh, W, V, ldw, targets);
  if (rc) return rc;
  if (T && dH && (rc = check_rows16(dH, dtype, d, lddh, "dH", false))) return rc;
  if (dW && (rc = check_rows16(dW, dtype, d, lddw, "dW", false))) return rc;
  if (T == 0) return dW ? launch_zero_rows(dW, dtype, V, (int)d, lddw, (hipStream_t)stream) : QAMW_OK;
  if (!aligned4(lse) || !aligned4(dloss)) return fail(QAMW_EINVAL, "lse and dloss must be non-NULL and 4-byte aligned");
  if (!dH && !dW) return QAMW_OK;
  const size_t need = qamw_cross_entropy_grad_workspace_bytes(T, V, d, dtype);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))
    return fail(QAMW_EWORKSPACE, "the cross entropy's gradient needs %zu bytes of 256-byte aligned workspace (got %zu)",
                need, workspace_bytes);
  return launch_cross_entropy_grad(H, dtype, T, (int)d, ldh, W, V, ldw, targets, lse, dloss, dH, lddh, dW, lddw,
                                   workspace, (hipStream_t)stream);
}

}  // extern "C"
