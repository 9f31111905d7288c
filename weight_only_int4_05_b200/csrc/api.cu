// api.cu -- the extern "C" entry points declared in include/awq_w4a16.h.
//
// Every entry point validates its arguments on the host and returns a status without launching
// anything when they are out of range; otherwise it enqueues the kernels on the caller's stream and
// returns.  No entry point allocates device memory.  The device status word (set by kernels whose
// bounded waits run out) is a file-scope __device__ variable; its address is looked up once per device.
#include <stdint.h>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"
#include "w8a8.cuh"

namespace awq {

__device__ unsigned g_device_status = 0u;

int num_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  if (cached[dev] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = v > 0 ? v : 1;
  }
  return cached[dev];
}

unsigned* device_status_ptr() {
  static unsigned* cached[64] = {nullptr};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  if (cached[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
    cached[dev] = static_cast<unsigned*>(p);
  }
  return cached[dev];
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxN = 1 << 21;   // sanity bounds on the sizes (a split linear further needs N / 32 <= 16384)
constexpr int kMaxK = 1 << 20;

static bool group_supported(int g) { return g == 64 || g == 128 || g == 256; }

awq_status check_linear(const uint16_t* x, const uint32_t* qw, const uint16_t* sc, const uint32_t* qz,
                               const uint16_t* y, int M, int N, int K, int g) {
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (M < 1 || N < 1 || K < g || K % g != 0 || N % 8 != 0 || N > kMaxN || K > kMaxK)
    return AWQ_ERR_INVALID_ARG;
  if (!x || !qw || !sc || !qz || !y) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(qw) || !aligned16(sc) || !aligned16(qz) || !aligned16(y))
    return AWQ_ERR_MISALIGNED;
  return AWQ_OK;
}

}  // namespace awq

using namespace awq;

extern "C" {

const char* awq_status_string(awq_status st) {
  switch (st) {
    case AWQ_OK: return "AWQ_OK";
    case AWQ_ERR_INVALID_ARG: return "AWQ_ERR_INVALID_ARG";
    case AWQ_ERR_UNSUPPORTED: return "AWQ_ERR_UNSUPPORTED";
    case AWQ_ERR_MISALIGNED: return "AWQ_ERR_MISALIGNED";
    case AWQ_ERR_CUDA: return "AWQ_ERR_CUDA";
    case AWQ_ERR_DEVICE_TIMEOUT: return "AWQ_ERR_DEVICE_TIMEOUT";
    case AWQ_ERR_WORKSPACE: return "AWQ_ERR_WORKSPACE";
    case AWQ_ERR_NUMERIC: return "AWQ_ERR_NUMERIC";
  }
  return "AWQ_ERR_UNKNOWN";
}

int awq_version(void) { return 100; }

awq_status awq_packed_sizes(int N, int K, int g, size_t* qweight_bytes, size_t* scales_bytes,
                            size_t* qzeros_bytes) {
  if (!qweight_bytes || !scales_bytes || !qzeros_bytes) return AWQ_ERR_INVALID_ARG;
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (N < 1 || K < 1 || K % g != 0 || N > kMaxN || K > kMaxK) return AWQ_ERR_INVALID_ARG;
  const size_t Np = (size_t)(N + 31) / 32 * 32;
  const size_t G = (size_t)K / (size_t)g;
  *qweight_bytes = Np * (size_t)K / 2;
  *scales_bytes = G * Np * 2;
  *qzeros_bytes = G * Np / 2;
  return AWQ_OK;
}

awq_status awq_act_scale(const uint16_t* d_xcal, int R, int K, uint16_t* d_s, awq_stream_t stream) {
  if (R < 1 || R > 8192 || K < 1 || K > kMaxK || !d_xcal || !d_s) return AWQ_ERR_INVALID_ARG;
  return prep_act_scale_launch(d_xcal, R, K, d_s, reinterpret_cast<cudaStream_t>(stream));
}

awq_status awq_apply_inv_scale(const uint16_t* d_x, const uint16_t* d_s, int M, int K, uint16_t* d_xp,
                               awq_stream_t stream) {
  if (M < 1 || K < 1 || K > kMaxK || !d_x || !d_s || !d_xp) return AWQ_ERR_INVALID_ARG;
  return prep_inv_scale_launch(d_x, d_s, M, K, d_xp, reinterpret_cast<cudaStream_t>(stream));
}

awq_status awq_pack(const uint16_t* d_W, const uint16_t* d_s, int N, int K, int g, uint32_t* d_qweight,
                    uint16_t* d_scales, uint32_t* d_qzeros, awq_stream_t stream) {
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (N < 1 || K < g || K % g != 0 || N > kMaxN || K > kMaxK) return AWQ_ERR_INVALID_ARG;
  if (!d_W || !d_qweight || !d_scales || !d_qzeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_W) || (d_s && !aligned16(d_s)) || !aligned16(d_qweight) || !aligned16(d_scales) ||
      !aligned16(d_qzeros))
    return AWQ_ERR_MISALIGNED;
  return pack_launch(d_W, nullptr, d_s, N, K, g, d_qweight, d_scales, d_qzeros, reinterpret_cast<cudaStream_t>(stream));
}

awq_status awq_pack_bits(const uint16_t* d_W, const uint16_t* d_s, int N, int K, int g, int w_bit, uint32_t* d_qweight,
                         uint16_t* d_scales, uint32_t* d_qzeros, awq_stream_t stream) {
  if (w_bit != 3 && w_bit != 4) return AWQ_ERR_UNSUPPORTED;
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (N < 1 || K < g || K % g != 0 || N > kMaxN || K > kMaxK) return AWQ_ERR_INVALID_ARG;
  if (!d_W || !d_qweight || !d_scales || !d_qzeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_W) || (d_s && !aligned16(d_s)) || !aligned16(d_qweight) || !aligned16(d_scales) ||
      !aligned16(d_qzeros))
    return AWQ_ERR_MISALIGNED;
  return pack_launch(d_W, nullptr, d_s, N, K, g, d_qweight, d_scales, d_qzeros, reinterpret_cast<cudaStream_t>(stream),
                     w_bit);
}

awq_status awq_packed3_sizes(int N, int K, int g, size_t* qweight_bytes, size_t* scales_bytes, size_t* qzeros_bytes) {
  awq_status st = awq_packed_sizes(N, K, g, qweight_bytes, scales_bytes, qzeros_bytes);
  if (st != AWQ_OK) return st;
  if (K % 32 != 0) return AWQ_ERR_INVALID_ARG;
  *qweight_bytes = *qweight_bytes / 4 * 3;  // 12 bytes per row per 32 channels instead of 16
  return AWQ_OK;
}

awq_status awq_pack3(const uint16_t* d_W, const uint16_t* d_s, int N, int K, int g, uint32_t* d_qweight,
                     uint16_t* d_scales, uint32_t* d_qzeros, awq_stream_t stream) {
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (N < 1 || K < g || K % g != 0 || N > kMaxN || K > kMaxK) return AWQ_ERR_INVALID_ARG;
  if (!d_W || !d_qweight || !d_scales || !d_qzeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_W) || (d_s && !aligned16(d_s)) || !aligned16(d_qweight) || !aligned16(d_scales) ||
      !aligned16(d_qzeros))
    return AWQ_ERR_MISALIGNED;
  return pack_launch(d_W, nullptr, d_s, N, K, g, d_qweight, d_scales, d_qzeros, reinterpret_cast<cudaStream_t>(stream),
                     3, 3);
}

awq_status awq_pack_gate_up(const uint16_t* d_Wgate, const uint16_t* d_Wup, const uint16_t* d_s, int NI, int K, int g,
                            uint32_t* d_qweight, uint16_t* d_scales, uint32_t* d_qzeros, awq_stream_t stream) {
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (NI < 16 || NI % 16 != 0 || 2 * (size_t)NI > (size_t)kMaxN || K < g || K % g != 0 || K > kMaxK)
    return AWQ_ERR_INVALID_ARG;
  if (!d_Wgate || !d_Wup || !d_qweight || !d_scales || !d_qzeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_Wgate) || !aligned16(d_Wup) || (d_s && !aligned16(d_s)) || !aligned16(d_qweight) ||
      !aligned16(d_scales) || !aligned16(d_qzeros))
    return AWQ_ERR_MISALIGNED;
  return pack_launch(d_Wgate, d_Wup, d_s, 2 * NI, K, g, d_qweight, d_scales, d_qzeros,
                     reinterpret_cast<cudaStream_t>(stream));
}

size_t w4a16_workspace_bytes(int mode, int M, int N, int K, int g) {
  if (!group_supported(g) || M < 1 || N < 1 || K < g || K % g != 0 || N % 8 != 0 || N > kMaxN || K > kMaxK)
    return SIZE_MAX;
  switch (mode) {
    case AWQ_MODE_GEMV: return gemv_workspace_bytes(M, N, K, g);
    case AWQ_MODE_GEMM: return gemm_workspace_bytes(M, N, K, g);
    case AWQ_MODE_LINEAR:
      return M <= w4a16_gemv_max_m(N, K) ? gemv_workspace_bytes(M, N, K, g) : gemm_workspace_bytes(M, N, K, g);
    default: return SIZE_MAX;
  }
}

static LinearArgs linear_args(const uint16_t* x, const uint32_t* qw, const uint16_t* sc, const uint32_t* qz,
                              uint16_t* y, int M, int N, int K, int g, void* ws, size_t ws_bytes, unsigned* status,
                              awq_stream_t stream) {
  LinearArgs a;
  a.x = x;
  a.qw = qw;
  a.scales = sc;
  a.qzeros = qz;
  a.y = y;
  a.M = M;
  a.N = N;
  a.K = K;
  a.g = g;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  a.status = status;
  a.st = reinterpret_cast<cudaStream_t>(stream);
  return a;
}

awq_status w4a16_gemv(const uint16_t* d_x, const uint32_t* d_qweight, const uint16_t* d_scales,
                      const uint32_t* d_qzeros, uint16_t* d_y, int M, int N, int K, int g, void* d_workspace,
                      size_t workspace_bytes, awq_stream_t stream) {
  awq_status st = check_linear(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g);
  if (st != AWQ_OK) return st;
  if (d_workspace && !aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  return gemv_launch(linear_args(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes,
                                 status, stream));
}

awq_status w4a16_gemv_s(const uint16_t* d_x, const uint16_t* d_s, const uint32_t* d_qweight,
                        const uint16_t* d_scales, const uint32_t* d_qzeros, uint16_t* d_y, int M, int N, int K, int g,
                        void* d_workspace, size_t workspace_bytes, awq_stream_t stream) {
  awq_status st = check_linear(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g);
  if (st != AWQ_OK) return st;
  if (d_s == nullptr) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_s) || (d_workspace && !aligned16(d_workspace))) return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  LinearArgs a = linear_args(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes,
                             status, stream);
  a.inv_s = d_s;
  return gemv_launch(a);
}

awq_status w4a16_gemm(const uint16_t* d_x, const uint32_t* d_qweight, const uint16_t* d_scales,
                      const uint32_t* d_qzeros, uint16_t* d_y, int M, int N, int K, int g, void* d_workspace,
                      size_t workspace_bytes, awq_stream_t stream) {
  awq_status st = check_linear(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g);
  if (st != AWQ_OK) return st;
  if (d_workspace && !aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  if (workspace_bytes < gemm_workspace_bytes(M, N, K, g)) return AWQ_ERR_WORKSPACE;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  return gemm_launch(linear_args(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes,
                                 status, stream));
}

// Crossover measured on B200 over the 70B-class shapes (M = 1 .. 256): the weight-streaming GEMV costs
// almost the same from M = 1 to 8 (one pass), 1.35x at M = 16 (two 8-row tiles per pass) and 2.7x at M = 32
// (two passes), and is faster than the tcgen05 GEMM through M = 32; from M = 64 the GEMM is faster.
int w4a16_gemv_max_m(int N, int K) {
  (void)N;
  (void)K;
  return 32;
}

awq_status w4a16_linear(const uint16_t* d_x, const uint32_t* d_qweight, const uint16_t* d_scales,
                        const uint32_t* d_qzeros, uint16_t* d_y, int M, int N, int K, int g, void* d_workspace,
                        size_t workspace_bytes, awq_stream_t stream) {
  if (M >= 1 && M <= w4a16_gemv_max_m(N, K))
    return w4a16_gemv(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes, stream);
  return w4a16_gemm(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes, stream);
}

awq_status w4a16_linear_pf(const uint16_t* d_x, const uint32_t* d_qweight, const uint16_t* d_scales,
                           const uint32_t* d_qzeros, uint16_t* d_y, int M, int N, int K, int g, void* d_workspace,
                           size_t workspace_bytes, const void* d_next, size_t next_bytes, awq_stream_t stream) {
  if (d_next == nullptr || next_bytes == 0 || M > w4a16_gemv_max_m(N, K))
    return w4a16_linear(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes, stream);
  if (!aligned16(d_next)) return AWQ_ERR_MISALIGNED;
  if (next_bytes % 16 != 0) return AWQ_ERR_INVALID_ARG;
  awq_status st = check_linear(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g);
  if (st != AWQ_OK) return st;
  if (d_workspace && !aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  LinearArgs a = linear_args(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes,
                             status, stream);
  a.pf = d_next;
  a.pf_bytes = next_bytes;
  return gemv_launch(a);
}

awq_status w4a16_gate_up_silu(const uint16_t* d_x, const uint32_t* d_qweight, const uint16_t* d_scales,
                              const uint32_t* d_qzeros, uint16_t* d_h, int M, int NI, int K, int g, void* d_workspace,
                              size_t workspace_bytes, awq_stream_t stream) {
  if (NI < 16 || NI % 16 != 0 || 2 * (size_t)NI > (size_t)kMaxN) return AWQ_ERR_INVALID_ARG;
  const int N = 2 * NI;
  awq_status st = check_linear(d_x, d_qweight, d_scales, d_qzeros, d_h, M, N, K, g);
  if (st != AWQ_OK) return st;
  if (d_workspace && !aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  LinearArgs a = linear_args(d_x, d_qweight, d_scales, d_qzeros, d_h, M, N, K, g, d_workspace, workspace_bytes,
                             status, stream);
  a.epi = 1;
  if (M <= w4a16_gemv_max_m(N, K)) return gemv_launch(a);
  if (workspace_bytes < gemm_workspace_bytes(M, N, K, g)) return AWQ_ERR_WORKSPACE;
  return gemm_launch(a);
}

awq_status w3a16_gemv(const uint16_t* d_x, const uint32_t* d_qweight, const uint16_t* d_scales,
                      const uint32_t* d_qzeros, uint16_t* d_y, int M, int N, int K, int g, void* d_workspace,
                      size_t workspace_bytes, awq_stream_t stream) {
  awq_status st = check_linear(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g);
  if (st != AWQ_OK) return st;
  if (d_workspace && !aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  LinearArgs a = linear_args(d_x, d_qweight, d_scales, d_qzeros, d_y, M, N, K, g, d_workspace, workspace_bytes,
                             status, stream);
  a.bits = 3;
  return gemv_launch(a);
}

static bool gptq_args_ok(int N, int K, int R, int g, double damp) {
  return N >= 1 && N % 8 == 0 && N <= kMaxN && K >= 128 && K % 128 == 0 && K % g == 0 && K <= 65536 && R >= 1 &&
         R <= (1 << 24) && damp >= 0.0;
}

size_t gptq_workspace_bytes(int N, int K, int R, int g) {
  if (!group_supported(g) || !gptq_args_ok(N, K, R, g, 0.0)) return SIZE_MAX;
  return awq::gptq_workspace_bytes(N, K);
}

awq_status gptq_quantize(const uint16_t* d_W, const uint16_t* d_xcal, int N, int K, int R, int g, double damp,
                         uint32_t* d_qweight, uint16_t* d_scales, uint32_t* d_qzeros, void* d_workspace,
                         size_t workspace_bytes, awq_stream_t stream) {
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (!gptq_args_ok(N, K, R, g, damp)) return AWQ_ERR_INVALID_ARG;
  if (!d_W || !d_xcal || !d_qweight || !d_scales || !d_qzeros) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_W) || !aligned16(d_xcal) || !aligned16(d_qweight) || !aligned16(d_scales) ||
      !aligned16(d_qzeros) || (d_workspace && !aligned16(d_workspace)))
    return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  return gptq_launch(d_W, d_xcal, N, K, R, g, damp, d_qweight, d_scales, d_qzeros, d_workspace, workspace_bytes,
                     status, reinterpret_cast<cudaStream_t>(stream));
}

static bool search_args_ok(int N, int K, int R, int g, int n_grid) {
  return N >= 1 && N % 8 == 0 && N <= kMaxN && K >= g && K % g == 0 && K <= kMaxK && R >= 1 && R <= 8192 &&
         n_grid >= 1 && n_grid <= 1000;
}

size_t awq_search_workspace_bytes(int N, int K, int R, int g, int n_grid) {
  if (!group_supported(g) || !search_args_ok(N, K, R, g, n_grid)) return SIZE_MAX;
  return search_workspace_bytes(N, K, R, g);
}

awq_status awq_search_scale(const uint16_t* d_W, const uint16_t* d_xcal, int N, int K, int R, int g, int n_grid,
                            double* d_losses, uint16_t* d_s, int32_t* d_best, void* d_workspace,
                            size_t workspace_bytes, awq_stream_t stream) {
  if (!group_supported(g)) return AWQ_ERR_UNSUPPORTED;
  if (!search_args_ok(N, K, R, g, n_grid)) return AWQ_ERR_INVALID_ARG;
  if (!d_W || !d_xcal || !d_losses || !d_s || !d_best) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_W) || !aligned16(d_xcal) || !aligned16(d_losses) || !aligned16(d_s) || !aligned16(d_best) ||
      (d_workspace && !aligned16(d_workspace)))
    return AWQ_ERR_MISALIGNED;
  unsigned* status = device_status_ptr();
  if (status == nullptr) return AWQ_ERR_CUDA;
  return search_launch(d_W, d_xcal, N, K, R, g, n_grid, d_losses, d_s, d_best, d_workspace, workspace_bytes, status,
                       reinterpret_cast<cudaStream_t>(stream));
}

// ---- 8-bit block-scaled operators
static bool dtype16(int dt) { return dt == AWQ_DTYPE_F16 || dt == AWQ_DTYPE_BF16; }
static bool size_ok(int v, int most, int multiple) { return v >= 1 && v <= most && v % multiple == 0; }

// CTAs write while others still read, and a workspace is written before the last read: an output or a workspace over anything
// else that the call takes is refused.
// Whether [a, a + na) and [b, b + nb) share a byte.
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

size_t fp8_scale_bytes(int R, int K) {
  if (!size_ok(R, 1 << 30, 1) || !size_ok(K, kMaxK, 16)) return SIZE_MAX;
  return (size_t)R * (size_t)fp8_scale_cols(K);
}

awq_status fp8_quantize(const void* d_x, int dtype, int R, int K, uint8_t* d_codes, uint8_t* d_scales,
                        awq_stream_t stream) {
  if (!dtype16(dtype)) return AWQ_ERR_UNSUPPORTED;
  if (!size_ok(R, 1 << 30, 1) || !size_ok(K, kMaxK, 16) || !d_x || !d_codes || !d_scales) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_x) || !aligned16(d_codes) || !aligned16(d_scales)) return AWQ_ERR_MISALIGNED;
  const size_t nx = (size_t)R * K * 2, nc = (size_t)R * K, ns = fp8_scale_bytes(R, K);
  if (overlap(d_codes, nc, d_x, nx) || overlap(d_scales, ns, d_x, nx) || overlap(d_codes, nc, d_scales, ns))
    return AWQ_ERR_INVALID_ARG;
  return fp8_quantize_launch(d_x, dtype, R, K, d_codes, d_scales, reinterpret_cast<cudaStream_t>(stream));
}

static awq_status check_w8a8(const void* x, const void* wc, const void* ws, const void* y, int dt, int M, int N, int K) {
  if (!dtype16(dt)) return AWQ_ERR_UNSUPPORTED;
  if (!size_ok(M, 1 << 24, 1) || !size_ok(N, kMaxN, 1) || !size_ok(K, kMaxK, 16)) return AWQ_ERR_INVALID_ARG;
  if (!x || !wc || !ws || !y) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(wc) || !aligned16(ws) || !aligned16(y)) return AWQ_ERR_MISALIGNED;
  return AWQ_OK;
}

static awq_status w8a8_product(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws, void* y,
                               int dt, int M, int N, int K, awq_stream_t stream, const uint16_t* x = nullptr) {
  W8Args a;
  a.x = x;
  a.xdt = dt;
  a.xc = xc;
  a.xs = xs;
  a.xrows = M;
  a.wc = wc;
  a.wsc = ws;
  a.N = N;
  a.K = K;
  a.y = y;
  a.dt = dt;
  a.status = device_status_ptr();
  a.st = reinterpret_cast<cudaStream_t>(stream);
  if (a.status == nullptr) return AWQ_ERR_CUDA;
  return w8a8_launch(a);
}

awq_status w8a8_gemm(const uint8_t* d_xcodes, const uint8_t* d_xscales, const uint8_t* d_wcodes,
                     const uint8_t* d_wscales, void* d_y, int dtype, int M, int N, int K, awq_stream_t stream) {
  awq_status st = check_w8a8(d_xcodes, d_wcodes, d_wscales, d_y, dtype, M, N, K);
  if (st != AWQ_OK) return st;
  if (!d_xscales) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_xscales)) return AWQ_ERR_MISALIGNED;
  const size_t ny = (size_t)M * N * 2;
  if (overlap(d_y, ny, d_xcodes, (size_t)M * K) || overlap(d_y, ny, d_xscales, fp8_scale_bytes(M, K)) ||
      overlap(d_y, ny, d_wcodes, (size_t)N * K) || overlap(d_y, ny, d_wscales, fp8_scale_bytes(N, K)))
    return AWQ_ERR_INVALID_ARG;
  return w8a8_product(d_xcodes, d_xscales, d_wcodes, d_wscales, d_y, dtype, M, N, K, stream);
}

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

size_t w8a8_workspace_bytes(int M, int N, int K) {
  if (!size_ok(M, 1 << 24, 1) || !size_ok(N, kMaxN, 1) || !size_ok(K, kMaxK, 16)) return SIZE_MAX;
  if (w8a8_quantizes(M)) return 0;  // the product quantizes few tokens itself
  return up256((size_t)M * K) + up256((size_t)M * fp8_scale_cols(K));
}

awq_status w8a8_linear(const void* d_x, int dtype, const uint8_t* d_wcodes, const uint8_t* d_wscales, void* d_y, int M,
                       int N, int K, void* d_workspace, size_t workspace_bytes, awq_stream_t stream) {
  awq_status st = check_w8a8(d_x, d_wcodes, d_wscales, d_y, dtype, M, N, K);
  if (st != AWQ_OK) return st;
  const size_t nx = (size_t)M * K * 2, ny = (size_t)M * N * 2, need = w8a8_workspace_bytes(M, N, K);
  if (need != 0 && (!d_workspace || workspace_bytes < need)) return AWQ_ERR_WORKSPACE;
  if (need != 0 && !aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  if (overlap(d_y, ny, d_x, nx) || overlap(d_y, ny, d_wcodes, (size_t)N * K) ||
      overlap(d_y, ny, d_wscales, fp8_scale_bytes(N, K)))
    return AWQ_ERR_INVALID_ARG;
  if (need != 0 && (overlap(d_workspace, need, d_x, nx) || overlap(d_workspace, need, d_y, ny) ||
                    overlap(d_workspace, need, d_wcodes, (size_t)N * K) ||
                    overlap(d_workspace, need, d_wscales, fp8_scale_bytes(N, K))))
    return AWQ_ERR_INVALID_ARG;
  if (w8a8_quantizes(M))
    return w8a8_product(nullptr, nullptr, d_wcodes, d_wscales, d_y, dtype, M, N, K, stream,
                        static_cast<const uint16_t*>(d_x));
  uint8_t* xc = static_cast<uint8_t*>(d_workspace);
  uint8_t* xs = xc + up256((size_t)M * K);
  st = fp8_quantize_launch(d_x, dtype, M, K, xc, xs, reinterpret_cast<cudaStream_t>(stream), true);
  if (st != AWQ_OK) return st;
  return w8a8_product(xc, xs, d_wcodes, d_wscales, d_y, dtype, M, N, K, stream);
}

awq_status moe_route(const void* d_logits, int dtype, const float* d_bias, int M, int E, int topk, int score, int groups,
                     int topk_groups, int renorm, float scale, int32_t* d_ids, float* d_weights, awq_stream_t stream) {
  if (!dtype16(dtype) && dtype != AWQ_DTYPE_F32) return AWQ_ERR_UNSUPPORTED;
  if (score != AWQ_SCORE_SOFTMAX && score != AWQ_SCORE_SIGMOID) return AWQ_ERR_UNSUPPORTED;
  if (!size_ok(M, 1 << 24, 1) || !size_ok(E, 1024, 1) || topk < 1 || topk > 32 || topk > E) return AWQ_ERR_INVALID_ARG;
  if (groups < 1 || groups > 32 || E % groups != 0 || topk_groups < 1 || topk_groups > groups ||
      topk > topk_groups * (E / groups))
    return AWQ_ERR_INVALID_ARG;
  if (!(scale == scale) || !d_logits || !d_ids || !d_weights) return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_logits) || (d_bias && !aligned16(d_bias)) || !aligned16(d_ids) || !aligned16(d_weights))
    return AWQ_ERR_MISALIGNED;
  const size_t nl = (size_t)M * E * (dtype == AWQ_DTYPE_F32 ? 4 : 2), nb = d_bias ? (size_t)E * 4 : 0,
               no = (size_t)M * topk * 4;
  if (overlap(d_ids, no, d_logits, nl) || overlap(d_weights, no, d_logits, nl) || overlap(d_ids, no, d_weights, no) ||
      (nb != 0 && (overlap(d_ids, no, d_bias, nb) || overlap(d_weights, no, d_bias, nb))))
    return AWQ_ERR_INVALID_ARG;
  return moe_route_launch(d_logits, dtype, d_bias, M, E, topk, score, groups, topk_groups, renorm, scale, d_ids,
                          d_weights, reinterpret_cast<cudaStream_t>(stream));
}

static bool moe_sizes_ok(int M, int E, int topk, int K, int I, int N) {
  return size_ok(M, 1 << 24, 1) && size_ok(E, 1024, 1) && topk >= 1 && topk <= 32 && (long long)M * topk <= (1 << 24) &&
         size_ok(K, kMaxK, 16) && size_ok(I, kMaxK, 16) && size_ok(N, kMaxN, 1) &&
         (long long)E * 2 * I <= (1 << 30) && (long long)E * N <= (1 << 30);
}

size_t w8a8_moe_workspace_bytes(int M, int E, int topk, int K, int I, int N) {
  if (!moe_sizes_ok(M, E, topk, K, I, N)) return SIZE_MAX;
  return moe_workspace_bytes(M, E, topk, K, I, N);
}

awq_status w8a8_moe(const void* d_x, int dtype, const int32_t* d_ids, const float* d_weights, const uint8_t* d_gu_codes,
                    const uint8_t* d_gu_scales, const uint8_t* d_down_codes, const uint8_t* d_down_scales, void* d_y,
                    int M, int E, int topk, int K, int I, int N, void* d_workspace, size_t workspace_bytes,
                    awq_stream_t stream) {
  if (!dtype16(dtype)) return AWQ_ERR_UNSUPPORTED;
  if (!moe_sizes_ok(M, E, topk, K, I, N)) return AWQ_ERR_INVALID_ARG;
  if (!d_x || !d_ids || !d_weights || !d_gu_codes || !d_gu_scales || !d_down_codes || !d_down_scales || !d_y)
    return AWQ_ERR_INVALID_ARG;
  if (!aligned16(d_x) || !aligned16(d_ids) || !aligned16(d_weights) || !aligned16(d_gu_codes) ||
      !aligned16(d_gu_scales) || !aligned16(d_down_codes) || !aligned16(d_down_scales) || !aligned16(d_y))
    return AWQ_ERR_MISALIGNED;
  if (!d_workspace || workspace_bytes < moe_workspace_bytes(M, E, topk, K, I, N)) return AWQ_ERR_WORKSPACE;
  if (!aligned16(d_workspace)) return AWQ_ERR_MISALIGNED;
  // y may be x: only the last kernel writes y, when x has been read.
  const size_t need = moe_workspace_bytes(M, E, topk, K, I, N), ny = (size_t)M * N * 2;
  const struct {
    const void* at;
    size_t bytes;
  } read[] = {{d_ids, (size_t)M * topk * 4},         {d_weights, (size_t)M * topk * 4},
              {d_gu_codes, (size_t)E * 2 * I * K},   {d_gu_scales, fp8_scale_bytes(E * 2 * I, K)},
              {d_down_codes, (size_t)E * N * I},     {d_down_scales, fp8_scale_bytes(E * N, I)}};
  if (overlap(d_workspace, need, d_y, ny) || overlap(d_workspace, need, d_x, (size_t)M * K * 2)) return AWQ_ERR_INVALID_ARG;
  for (const auto& r : read)
    if (overlap(d_y, ny, r.at, r.bytes) || overlap(d_workspace, need, r.at, r.bytes)) return AWQ_ERR_INVALID_ARG;
  MoeArgs a;
  a.x = static_cast<const uint16_t*>(d_x);
  a.ids = d_ids;
  a.weights = d_weights;
  a.guc = d_gu_codes;
  a.gus = d_gu_scales;
  a.dc = d_down_codes;
  a.ds = d_down_scales;
  a.y = static_cast<uint16_t*>(d_y);
  a.dt = dtype;
  a.M = M;
  a.E = E;
  a.topk = topk;
  a.K = K;
  a.I = I;
  a.N = N;
  a.ws = d_workspace;
  a.status = device_status_ptr();
  a.st = reinterpret_cast<cudaStream_t>(stream);
  if (a.status == nullptr) return AWQ_ERR_CUDA;
  return moe_launch(a);
}

awq_status awq_last_device_status(awq_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return AWQ_ERR_CUDA;
  unsigned* p = device_status_ptr();
  if (p == nullptr) return AWQ_ERR_CUDA;
  unsigned v = 0u;
  if (cudaMemcpy(&v, p, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return AWQ_ERR_CUDA;
  if (v != 0u) {
    const unsigned zero = 0u;
    if (cudaMemcpy(p, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess) return AWQ_ERR_CUDA;
    return v == 2u ? AWQ_ERR_NUMERIC : AWQ_ERR_DEVICE_TIMEOUT;
  }
  return AWQ_OK;
}

}  // extern "C"
