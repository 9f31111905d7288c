// fp8.cu -- fp8_quantize: a 16-bit matrix to e4m3 codes with one power-of-two scale per row and 128 columns.
//
// Bound by memory: 2 bytes read and 1 + 1/128 written per value.  14336 x 4096 takes 28.7 us, 6.1 TB/s, 94 % of the measured
// copy rate.  Measured on the way: the item number split by a 64-bit division, 43 us (the division took longer than the
// quantizing); 32-bit steps with the next item's loads ahead, 28.7 us.
#include "fp8.cuh"

namespace awq {

// EARLY: dependents may start at once, for the caller who quantizes activations and whose next kernel waits before it reads
// them; a weight's quantizer never signals early, so that a product behind it may prefetch weights ahead of its wait.
// One warp takes 512 columns of one row: lane l holds the 8 columns at 8 l of each half (two 16-byte loads), so the
// 16 lanes of a half warp share a block of 128 and its maximum takes four shuffles; the four scale bytes are one word.
template <int DT, bool EARLY>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const uint16_t* x, int R, int K, int SW, uint8_t* codes,
                                                           uint32_t* scales) {
  if (EARLY) pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int step = (int)gridDim.x * 8, first = (int)blockIdx.x * 8 + (int)(threadIdx.x >> 5);
  const int step_row = step / SW, step_w = step - step_row * SW;  // one division each here instead of one per item
  int row = first / SW, w = first - row * SW;
  const int blocks = fp8_blocks(K);
  uint4 v[2];
  auto load = [&](int r, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = c * 512 + h * 256 + lane * 8;
      v[h] = make_uint4(0u, 0u, 0u, 0u);
      if (r < R && k < K) v[h] = ldg_stream(x + (size_t)r * K + k);
    }
  };
  load(row, w);
  while (row < R) {
    const uint4 now[2] = {v[0], v[1]};
    int next_row = row + step_row, next_w = w + step_w;
    if (next_w >= SW) {
      next_w -= SW;
      ++next_row;
    }
    load(next_row, next_w);  // the next item's values are on their way while this one is quantized
    uint32_t word = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u[4] = {now[h].x, now[h].y, now[h].z, now[h].w};
      float f[8];
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = pair_to_f32<DT>(u[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
        m = fmaxf(m, fmaxf(fabsf(p.x), fabsf(p.y)));
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      const uint32_t b = fp8_scale_byte(__float_as_uint(m));
      const float inv = fp8_inv_scale(b);
      const int k = w * 512 + h * 256 + lane * 8;
      if (k < K) {
        uint2 c;
        c.x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
        c.y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
        *reinterpret_cast<uint2*>(codes + (size_t)row * K + k) = c;
      }
      const int blk = w * 4 + h * 2;
      const uint32_t other = __shfl_sync(0xFFFFFFFFu, b, 16);  // the second block of this half, for lane 0
      word |= (blk < blocks ? b : 127u) << (16 * h);
      word |= (blk + 1 < blocks ? other : 127u) << (16 * h + 8);
    }
    if (lane == 0) scales[(size_t)row * SW + w] = word;
    row = next_row;
    w = next_w;
  }
}

awq_status fp8_quantize_launch(const void* x, int dt, int R, int K, uint8_t* codes, uint8_t* scales, cudaStream_t st,
                               bool early) {
  const int SW = fp8_scale_cols(K) / 4;
  const long long warps = (long long)R * SW;
  long long blocks = (warps + 7) / 8;
  const long long cap = (long long)num_sms() * 8;
  if (blocks > cap) blocks = cap;
  auto kernel = dt == AWQ_DTYPE_F16
                    ? (early ? fp8_quantize_kernel<AWQ_DTYPE_F16, true> : fp8_quantize_kernel<AWQ_DTYPE_F16, false>)
                    : (early ? fp8_quantize_kernel<AWQ_DTYPE_BF16, true> : fp8_quantize_kernel<AWQ_DTYPE_BF16, false>);
  cudaError_t e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, st, static_cast<const uint16_t*>(x), R, K, SW,
                             codes, reinterpret_cast<uint32_t*>(scales));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
