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

// silu(a) = a / (1 + e^-a) to 2^-20 of it (2^-119 where it is smaller than that), for every a: its limits a and 0 at the ends,
// NaN for NaN.  e^-a = 2^(hi + lo), -a log2(e) carried in two parts (the argument reduction of Cody and Waite, "Software Manual
// for the Elementary Functions", 1980, with base 2), since hi alone is off by up to 126 * 2^-24.
// Past |hi| = 126 lo does not count: below it e is 0, or lost beside 1; above it silu is 0 to 2^-119.  There lo may be infinite or
// NaN (hi overflows from |a| = 2.36e38 on, and a itself may be infinite), and so may e.
__device__ __forceinline__ float fp8_silu(float a) {
  const float hi = -a * 1.44269504f;
  const float lo = fmaf(-a, 1.44269504f, -hi) - a * 1.92596299e-8f;
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(hi));
  if (fabsf(hi) < 126.f) e = fmaf(e, lo * 0.693147181f, e);
  return __fdividef(hi >= 126.f ? 0.f : a, 1.0f + e);
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

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in CTA `rank` of the cluster, of the shared variable at `p` in this one.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// A whole warp waits for the phase with the given parity; all lanes get the same answer.  False after kWaitLimitNs
// (recorded in *status) or once another role of the CTA gave up; either way *abort_flag is set.  CLUSTER: acquire what other
// CTAs of the cluster wrote before they arrived, for this warp's own loads (several hundred cycles more per wait).
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, unsigned* status, volatile int* abort_flag) {
  auto passed = [&]() {
    return __all_sync(0xFFFFFFFFu, CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity));
  };
  if (passed()) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (unsigned it = 0;; ++it) {
    if (passed()) return true;
    if ((it & 63u) == 63u) {
      const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
      if (__any_sync(0xFFFFFFFFu, late || *abort_flag)) {
        if (late) atomicExch(status, kDevTimeout);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// ---------------------------------------------------------------- tcgen05, block-scaled, one CTA or a pair (CG)
// D[tmem] (+)= (A 2^sfa) (B 2^sfb)^T for one K step of 32 e4m3 codes, fp32 sums; the scales are bytes of 32-bit
// words in tensor memory (row r of A: lane r % 32, column r / 32), the byte chosen in the instruction descriptor.
template <int CG>
__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}
// 32 rows of 16 bytes from shared memory into 4 tensor-memory columns, repeated in the four 32-lane quarters (a pair:
// each CTA from its own shared memory).
template <int CG>
__device__ __forceinline__ void tmem_cp_32x128(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Arrive on `bar` (a pair: at the same place in both CTAs) when every tcgen05 operation issued so far has completed.
template <int CG>
__device__ __forceinline__ void umma_commit_group(uint64_t* bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_group(uint32_t* dst_smem, unsigned ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_group(uint32_t taddr, unsigned ncols) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// 2-D tensor copy into this CTA's shared memory, completing on a barrier given by its cluster address (a pair: the
// even CTA's).
template <int CG>
__device__ __forceinline__ void tma_load_2d_group(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
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
