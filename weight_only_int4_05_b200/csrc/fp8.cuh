// fp8.cuh -- device helpers of the 8-bit block-scaled operators (fp8.cu, w8a8.cu, moe.cu).
//
// An 8-bit matrix X [R][K] is e4m3 codes [R][K] and one power-of-two scale (e8m0 byte b: 2^(b - 127)) per row
// and block of 128 columns, [R][SC] bytes with SC = ceil(K / 128) rounded up to a multiple of 4, so that the four
// scales of 512 columns are one 32-bit word.  The scale of a block is the smallest power of two 2^t >= 2^-126 with
// max|x| <= 448 * 2^t (448 is e4m3's largest value); a code is x * 2^-t rounded to nearest even.  Every step but
// that rounding is exact, so the codes do not depend on how a kernel is written.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace awq {

constexpr int kFp8Block = 128;  // columns that share a scale

__host__ __device__ constexpr int fp8_blocks(int K) { return (K + kFp8Block - 1) / kFp8Block; }
__host__ __device__ constexpr int fp8_scale_cols(int K) { return (fp8_blocks(K) + 3) / 4 * 4; }

// The e8m0 byte of a block from the bits of its largest magnitude: amax = m 2^p (1 <= m < 2) needs t = p - 8 when
// m <= 1.75 and p - 7 otherwise (448 = 1.75 * 2^8); blocks below 448 * 2^-126 (a block of zeros among them) take 2^-126.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits) {
  const int b = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(b < 1 ? 1 : b);
}
// 2^(127 - b) = 1 / 2^(b - 127): multiplying by it is exact.  b is 1 .. 248 here, so the exponent field is normal.
__device__ __forceinline__ float fp8_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two values to two e4m3 codes (lo in the low byte), to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- 16-bit types
template <int DT>
__device__ __forceinline__ float2 pair_to_f32(uint32_t v) {
  if constexpr (DT == AWQ_DTYPE_F16) {
    return __half22float2(*reinterpret_cast<__half2*>(&v));
  } else {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
}
// One fp32 value rounded to the type's 16 bits (round to nearest even).
__device__ __forceinline__ uint16_t f32_to_16(float v, int dt) {
  return dt == AWQ_DTYPE_F16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// ---------------------------------------------------------------- tcgen05, block-scaled
// D[tmem] (+)= (A * 2^sfa) (B * 2^sfb)^T for one K step of 32 e4m3 codes, fp32 sums; the scales are bytes of 32-bit
// words in tensor memory (row r of A: lane r % 32, column r / 32), the byte chosen in the instruction descriptor.
__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}
// 32 rows of 16 bytes from shared memory into 4 tensor-memory columns, repeated in the four 32-lane quarters.
__device__ __forceinline__ void tmem_cp_32x128(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Descriptor of 512 contiguous bytes read as 32 rows of 16 (8-row core matrices of 128 bytes, no swizzle).
__device__ __forceinline__ uint64_t umma_desc_plain(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);  // start address >> 4
  d |= (uint64_t)(16u >> 4) << 16;               // leading byte offset (one core matrix along K: unused)
  d |= (uint64_t)(128u >> 4) << 32;              // stride byte offset: next 8 rows
  d |= (uint64_t)1 << 46;                        // descriptor version for sm_100
  return d;
}
// Instruction descriptor: kind::mxf8f6f4, A = B = e4m3, both K-major, e8m0 scales, M x N tile, scale bytes 0.
__host__ __device__ constexpr uint32_t umma_idesc_mxf8(int M, int N) {
  return (0u << 7) | (0u << 10)           // A, B e4m3
         | ((uint32_t)(N >> 3) << 17)     // N / 8
         | (1u << 23)                     // scales e8m0
         | ((uint32_t)(M >> 7) << 27);    // M / 128
}
// The same descriptor reading byte `sf` (0..3) of both scale words.
__device__ __forceinline__ uint32_t umma_idesc_sf(uint32_t idesc, uint32_t sf) { return idesc | (sf << 4) | (sf << 29); }

}  // namespace awq
