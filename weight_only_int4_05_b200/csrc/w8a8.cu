// w8a8.cu -- the product of two 8-bit block-scaled matrices on the tcgen05 tensor cores.
//
// y^T tile [128 weight rows][BT tokens] = sum over blocks of 128 channels of (C_w T_w) . (C_x T_x)^T, with e4m3 codes C and
// power-of-two scales T.  The scales go to tensor memory beside the accumulator and the tensor cores apply them
// (kind::mxf8f6f4.block_scale): one scale byte serves the four 32-channel steps of its block, so a block of 128 costs
// the same as the format's native 32 and no partial sum leaves tensor memory.  Weights are the A operand (128 rows of
// N), tokens the B operand, so a few tokens still fill the instruction's height.
//
// Per CTA (12 warps), persistent over output tiles, k-blocks of 128 channels through an ST-stage ring:
//   warp 0      producer: TMA copies of the weight rows and of the tokens (128-byte swizzle) onto full[s].
//   warp 1      MMA: per k-block 4 x tcgen05.mma (32 channels each); every 4th k-block first copies the next scale words
//               from shared to tensor memory (tcgen05.cp).
//   warps 2, 3  scales: one 32-bit word per row holds the scales of 4 k-blocks; they fill the slots in turn.
//   warps 4..11 epilogue, two warpgroups taking 16 tokens (a lone CTA's: 4) in turn: tensor memory -> registers -> y, or
//               h = silu(gate) up quantized again.
// What bounds it and what each part measured (us, B200):
//   2048 x 28672 x 8192: the tensor cores, then the 1000 W cap (the SM clock falls to 1.2 - 1.5 GHz): 360 - 445, 2.2 - 2.7
//     PFLOP/s by the card, the tensor pipe active 79 % of all cycles; 718 with one CTA per tile and one accumulator, whose
//     epilogue nothing covered.
//   16 x 14336 x 4096: the weight's bytes, 16.7 (3.6 TB/s; they would take 9.2, the rest goes to the way from x to the first
//     product, the joining of the parts and the hand-over between kernels, during which only the next kernel's first ring is
//     fetched).
//   1 x 4096 x 4096: latency, 8.4; 26 when 32 CTAs each took the whole of K, 8.7 when the parts were fetched instead of sent.
//   gate|up and down of 64 experts (4096/1024), 2048 tokens top 6: 114 and 95 - 101, 5.3 and 4.8 - 5.1 TB/s of weights and rows.
// Two accumulators alternate, so a tile's epilogue runs under the next tile's products; where two do not fit beside the
// scales they share some columns, which the epilogue reads first.
// Many tokens (CG = 2): two CTAs work on one tile of 256 weight rows; each holds its 128 rows, half of the tokens' codes and
// its half of the accumulator, so each byte of x brought to an SM serves 256 rows.
// Few tokens (splits > 1): a cluster shares one tile, each CTA a part of K; each CTA finishes some of the tokens, whose parts
// the others put into its shared memory and it sums in rank order, so there is no workspace and no counter.
// At most 16 tokens (XQ): x comes as 16-bit values and the epilogue warps, idle until the tile's products are done,
// quantize it into the ring, each CTA the part of K that it needs, so a decode step has no quantizer launch in front of it;
// the codes and scales are those of fp8_quantize, bit for bit.
// Every mbarrier wait is bounded; a timeout is recorded in the status word, the CTA drains its copies and MMAs, frees
// its tensor memory and exits.
#include <math.h>

#include <type_traits>

#include "fp8.cuh"
#include "w8a8.cuh"

namespace awq {

namespace {

constexpr int kTileW = 128;        // weight rows per accumulator and CTA
constexpr int kBlkBytes = 128;     // bytes of K per k-block: one swizzle row, one scale block
template <int CG>
constexpr int kEpi = 2;  // epilogue warpgroups
// Tokens up to which the epilogue warps quantize x: 8 warps of 2 rows.  16 x 14336 x 4096 takes 16.7 us, 17.6 with the quantizer
// in front, and a call one launch and no scratch instead of two and some (13 instead of 20 us on the host); passes over up to
// 64 rows were slower than the quantizer in front (333 x 1000 x 1040: 13.5 against 9.0 us).
constexpr int kXqMost = 16;
// k-blocks per part of a split K: joining parts takes about as long as 8 of them (1 x 4096 x 4096 takes as long in 4 parts of 8
// as in 8 parts of 4; 9 k-blocks of an expert's gate|up took 19 us in 2 parts and 15.7 whole).
constexpr int kPartLeast = 8;
// Accumulator columns up to which a CTA takes half an SM's shared memory: one token over two of eight 4096/14336 experts, 88 us
// with whole SMs, 75 with halves.  With 64 columns of gate|up (two weight tiles of 16 KB per stage) a half holds two stages only.
constexpr int kHalfMost = 32;
template <int CG>
constexpr int kW8Threads = 128 + 128 * kEpi<CG>;
constexpr int kW8Smem = 232448;    // opt-in dynamic shared memory per block on sm_100
constexpr int kW8HalfSmem = 115712;  // two blocks per SM (1 KB of each block's share is the system's)
constexpr int kSplitMost = 64;     // tokens per tile up to which K is split (64 x 4096 x 14336: 38 us whole, 20 split)
constexpr int kPairLeast = 64;     // tokens per tile from which two CTAs work on it together (112: 151 us alone, 136 paired)
template <bool XQ>
constexpr int kSf = XQ ? 2 : 4;    // scale slots (4 k-blocks each) in shared memory
constexpr int kSfTmem = 2;         // and in tensor memory

struct W8Params {
  const uint32_t* ws;  // scale words of w and x, SW per row
  const uint32_t* xs;
  const uint16_t* x;   // XQ: x itself, [xrows][K] of type xdt
  int K, xdt, plan_ready;
  void* y;
  uint8_t* hc;
  uint8_t* hs;
  const int* row_start;
  const int* tile_start;
  unsigned* status;
  int xrows, wrows, wtotal;  // rows of x, weight rows per group, weight rows in all
  int N, KB, SW, SWh;
  int BT, ST, tmem_cols, acc_off, groups, n_tiles, t_tiles, splits, dt;
  uint32_t idesc;
};

struct W8Tile {
  int w0, n0, t0, rows;  // first weight row (in the stack of all groups), first output, first token row, valid token rows
};

template <int EPI>
constexpr int kAtomsA = EPI == kW8SiluQuant ? 2 : 1;  // accumulators (weight row sets) per tile

__host__ __device__ constexpr int w8_stage(int atoms, int x_rows) { return (atoms * kTileW + x_rows) * kBlkBytes; }
__host__ __device__ constexpr int w8_sf_slot(int atoms, int BT) { return (atoms + (BT + 127) / 128) * 512; }
__host__ __device__ constexpr int w8_sf_cols(int atoms, int BT) { return (atoms + (BT + 127) / 128) * 4; }

// Tile number -> place; a tile is 128 * CG weight rows.  Dense: token tiles fastest, so the tiles in flight share weight
// rows.  Grouped: group by group, token tiles fastest within a weight tile; tabs = [tile_start | row_start].
template <int CG>
__device__ __forceinline__ W8Tile w8_tile(const W8Params& p, const int* tabs, int tile, int rank) {
  W8Tile r;
  if (p.groups == 0) {
    const int n = tile / p.t_tiles, t = tile - n * p.t_tiles;
    r.n0 = n * (kTileW * CG) + (CG == 2 ? rank * kTileW : 0);
    r.w0 = r.n0;
    r.t0 = t * p.BT;
    r.rows = min(p.BT, p.xrows - r.t0);
    return r;
  }
  int lo = 0, hi = p.groups - 1;  // the last group whose first tile is not behind `tile` (empty groups have no tiles)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tabs[mid] * p.n_tiles <= tile) lo = mid; else hi = mid - 1;
  }
  const int tt = tabs[lo + 1] - tabs[lo];
  const int local = tile - tabs[lo] * p.n_tiles;
  const int n = local / tt, t = local - n * tt;
  const int* rows = tabs + p.groups + 1;
  r.n0 = n * (kTileW * CG) + (CG == 2 ? rank * kTileW : 0);
  r.w0 = lo * p.wrows + r.n0;
  r.t0 = rows[lo] + t * p.BT;
  r.rows = min(p.BT, rows[lo + 1] - r.t0);
  return r;
}

struct W8Maps {
  CUtensorMap w, x;
};

// W columns of this warp's 32 lanes of tensor memory; the registers hold them after tmem_wait_ld alone.
template <int W>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[W]) {
  if constexpr (W == 16) {
    tmem_ld_32x32b_x16(taddr, v);
  } else {
    static_assert(W == 4, "4 or 16 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(taddr)
                 : "memory");
  }
}
template <int W>
__device__ __forceinline__ void tmem_cols_f32(const uint32_t (&v)[W], float (&f)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) f[i] = __uint_as_float(v[i]);
}

// Outputs of weight row n0 + row for the W tokens from column c of the tile on.
template <int W, typename T, typename F>
__device__ __forceinline__ void w8_store_as(const W8Params& p, const W8Tile& t, int row, int c, const float (&f)[W], F to) {
  T* y = static_cast<T*>(p.y) + (size_t)(t.t0 + c) * p.N + (t.n0 + row);
  const int rows = t.rows - c;
  if (rows >= W) {
#pragma unroll
    for (int i = 0; i < W; ++i, y += p.N) *y = to(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i, y += p.N)
      if (i < rows) *y = to(f[i]);
  }
}
template <int W>
__device__ __forceinline__ void w8_store(const W8Params& p, const W8Tile& t, int row, int c, const float (&f)[W]) {
  if (t.n0 + row >= p.N) return;
  if (p.dt == AWQ_DTYPE_F32)
    w8_store_as<W, float>(p, t, row, c, f, [](float v) { return v; });
  else if (p.dt == AWQ_DTYPE_F16)
    w8_store_as<W, __half>(p, t, row, c, f, [](float v) { return __float2half_rn(v); });
  else
    w8_store_as<W, __nv_bfloat16>(p, t, row, c, f, [](float v) { return __float2bfloat16_rn(v); });
}

// The same through shared memory, for the pair's large tiles: 16 tokens of the 128 rows are turned round, so that a warp
// writes whole runs of 128 outputs of 4 tokens (256 or 512 contiguous bytes) where it wrote 16 runs of 32; for outputs whose
// row length is a multiple of 4.  `turned` is the warpgroup's [16][128]; v gets the 4 outputs of tokens 4 q .. 4 q + 3 from
// output 4 lane on.  Written straight from the registers the quantizing epilogue below took 24000 cycles per
// tile of 112 tokens, this way 14000, and gate|up of the experts 118 us instead of 135.  A bulk copy per token from
// shared memory in place of the wide stores was slower (the experts' down projection: 121 us against 95).
__device__ __forceinline__ void w8_turn(const float (&f)[16], int row, uint32_t turned, int bar, float4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(turned + (uint32_t)(i * kTileW + row) * 4), "f"(f[i]) : "memory");
  named_barrier_sync(bar, 128);
  const uint32_t src = turned + (uint32_t)((row >> 5) * (4 * kTileW) + (row & 31) * 4) * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[j].x), "=f"(v[j].y), "=f"(v[j].z), "=f"(v[j].w)
                 : "r"(src + j * kTileW * 4)
                 : "memory");
  named_barrier_sync(bar, 128);
}
__device__ __forceinline__ void st_global_v2(void* p, uint32_t a, uint32_t b) {
  asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void w8_put(float* y, float4 v) {
  asm volatile("st.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(y), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void w8_put(__half* y, float4 v) {
  st_global_v2(y, h2_as_u32(__floats2half2_rn(v.x, v.y)), h2_as_u32(__floats2half2_rn(v.z, v.w)));
}
__device__ __forceinline__ void w8_put(__nv_bfloat16* y, float4 v) {
  __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  st_global_v2(y, *reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
}
template <typename T>
__device__ __forceinline__ void w8_store_turned_as(const W8Params& p, const W8Tile& t, int row, int c, const float4 (&v)[4]) {
  const int n = t.n0 + (row & 31) * 4, first = c + (row >> 5) * 4, rows = t.rows - first;
  if (n >= p.N) return;
  T* y = static_cast<T*>(p.y) + (size_t)(t.t0 + first) * p.N + n;
#pragma unroll
  for (int j = 0; j < 4; ++j, y += p.N)
    if (j < rows) w8_put(y, v[j]);
}
__device__ __forceinline__ void w8_store_turned(const W8Params& p, const W8Tile& t, int row, int c, const float (&f)[16],
                                                uint32_t turned, int bar) {
  float4 v[4];
  w8_turn(f, row, turned, bar, v);
  if (p.dt == AWQ_DTYPE_F32) w8_store_turned_as<float>(p, t, row, c, v);
  else if (p.dt == AWQ_DTYPE_F16) w8_store_turned_as<__half>(p, t, row, c, v);
  else w8_store_turned_as<__nv_bfloat16>(p, t, row, c, v);
}

// h = silu(a) b of 16 tokens, quantized, through shared memory as above: a warp holds the 128 channels of a token, one block
// of the 8-bit format, 4 per lane.
__device__ __forceinline__ void w8_silu_quant_turned(const W8Params& p, const W8Tile& t, int row, int c,
                                                     const float (&a)[16], const float (&b)[16], uint32_t turned, int bar) {
  const int lane = row & 31, n = t.n0 + lane * 4, first = c + (row >> 5) * 4, rows = t.rows - first;
  float h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = fp8_silu(a[i]) * b[i];
  if (t.n0 + row >= p.N) {  // rows of another expert or of none
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = 0.f;
  }
  float4 v[4];
  w8_turn(h, row, turned, bar, v);
  uint32_t s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float m = fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)), fmaxf(fabsf(v[j].z), fabsf(v[j].w)));
    s[j] = fp8_scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m)));
  }
  uint8_t* hc = p.hc + (size_t)(t.t0 + first) * p.N + n;
  uint8_t* hs = p.hs + (size_t)(t.t0 + first) * (p.SWh * 4) + t.n0 / kFp8Block;
#pragma unroll
  for (int j = 0; j < 4; ++j, hc += p.N, hs += p.SWh * 4) {
    const float inv = fp8_inv_scale(s[j]);
    const uint32_t q = e4m3x2(v[j].x * inv, v[j].y * inv) | (e4m3x2(v[j].z * inv, v[j].w * inv) << 16);
    // N is a multiple of 16
    if (j < rows && n < p.N) asm volatile("st.global.b32 [%0], %1;" ::"l"(hc), "r"(q) : "memory");
    if (j < rows && lane == 0) asm volatile("st.global.b8 [%0], %1;" ::"l"(hs), "r"(s[j]) : "memory");
  }
}

// h = silu(a) b of the same tokens, quantized: the 128 rows of the tile are one block of the 8-bit format, so its maximum
// is taken over the four warps of a warpgroup.  `amax` [2][4][16] alternates by `turn`, so one barrier per call is enough.
template <int W>
__device__ __forceinline__ void w8_silu_quant(const W8Params& p, const W8Tile& t, int row, int c, const float (&a)[W],
                                              const float (&b)[W], uint32_t* amax, int& turn, int bar) {
  const int n = t.n0 + row, lane = row & 31, q = row >> 5;
  uint32_t* buf = amax + turn * 64;
  turn ^= 1;
  float h[W];
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    h[i] = n < p.N ? fp8_silu(a[i]) * b[i] : 0.f;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h[i])));
    if (lane == i) mine = m;
  }
  if (lane < W) buf[q * 16 + lane] = mine;
  named_barrier_sync(bar, 128);
  uint8_t* hc = p.hc + (size_t)(t.t0 + c) * p.N + n;
  uint8_t* hs = p.hs + (size_t)(t.t0 + c) * (p.SWh * 4) + t.n0 / kFp8Block;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t s = fp8_scale_byte(max(max(buf[i], buf[16 + i]), max(buf[32 + i], buf[48 + i])));
    if (c + i < t.rows && n < p.N) {
      hc[(size_t)i * p.N] = (uint8_t)e4m3x2(h[i] * fp8_inv_scale(s), 0.f);
      if (row == 0) hs[i * (p.SWh * 4)] = (uint8_t)s;
    }
  }
}

// One tile's x into its own ring (XQ): warp xw takes token rows 2 xw and 2 xw + 1, half a warp per row, 8 values per lane and
// k-block.  Four k-blocks go at a time, the loads of the next four behind them; their codes stand in slot cs of `xring`
// beside the slot's scale words, so that one wait and one arrival serve all (with the codes in the weight's stages it
// took five of each, 200 to 350 cycles apiece on the way from x to the first product: 1 x 4096 x 4096 9.4 us, now 8.7).
struct XqState {
  int cs = 0;  // scale slot
  unsigned phase = 1;
};
template <int DT>
__device__ __forceinline__ void w8_quantize_x(const W8Params& p, const W8Tile& t, uint8_t* xring, uint8_t* sfx, int slot,
                                              uint64_t* sf_full, uint64_t* sf_empty, volatile int* abort_flag, int kb0,
                                              int kb1, int xw, int lane, XqState& st) {
  const int r = xw * 2 + (lane >> 4);
  const uint16_t* x = p.x + (size_t)(t.t0 + min(r, t.rows - 1)) * p.K + (lane & 15) * 8;
  const int last = r < t.rows ? p.K - (lane & 15) * 8 : 0;  // columns from here on exist (in steps of 8)
  // 128-byte swizzle: 16-byte piece n of row r stands at piece n ^ (r % 8)
  uint8_t* to = xring + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8;
  uint4 v[4];
  auto load = [&](int c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kb = 4 * c + j;
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (kb >= kb0 && kb < kb1 && kb * kFp8Block < last) v[j] = *reinterpret_cast<const uint4*>(x + kb * kFp8Block);
    }
  };
  const int c1 = (kb1 + 3) >> 2;
  load(kb0 >> 2);
  for (int c = kb0 >> 2; c < c1; ++c) {
    uint2 q[4];
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      float f[8], m = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 pr = pair_to_f32<DT>(u[k]);
        f[2 * k] = pr.x;
        f[2 * k + 1] = pr.y;
        m = fmaxf(m, fmaxf(fabsf(pr.x), fabsf(pr.y)));
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      const uint32_t b = fp8_scale_byte(__float_as_uint(m));
      const float inv = fp8_inv_scale(b);
      word |= b << (8 * j);
      q[j].x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
      q[j].y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
    }
    if (c + 1 < c1) load(c + 1);
    if (!warp_wait(&sf_empty[st.cs], st.phase, p.status, abort_flag)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint2*>(to + (st.cs * 4 + j) * (16 * kBlkBytes)) = q[j];
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(sfx + st.cs * slot + r * 16) = word;  // rows 0 .. 31: the first word of 16 bytes
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sf_full[st.cs]);
    if (++st.cs == kSf<true>) {
      st.cs = 0;
      st.phase ^= 1u;
    }
  }
}

}  // namespace

template <int EPI, int CG, bool XQ>
__global__ void __launch_bounds__(kW8Threads<CG>, CG == 1 ? 2 : 1) w8a8_kernel(const __grid_constant__ W8Maps maps, const W8Params p) {
  constexpr int NA = kAtomsA<EPI>;
  extern __shared__ uint8_t w8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(w8_smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage = w8_stage(NA, XQ ? 0 : p.BT / CG), slot = w8_sf_slot(NA, p.BT);
  uint8_t* sf = smem + p.ST * stage;
  uint8_t* xring = sf + kSf<XQ> * slot;  // XQ: the codes of x, 4 k-blocks of 16 rows per scale slot
  float* part = reinterpret_cast<float*>(xring + (XQ ? kSf<XQ> * 4 * 16 * kBlkBytes : 0));  // splits > 1: [NA * BT][128] partial sums
  // a pair: [kEpi][16][128], the epilogue's turning space in its place
  uint64_t* full = reinterpret_cast<uint64_t*>(part + (CG == 2 ? kEpi<CG> * 16 * kTileW : p.splits > 1 ? NA * p.BT * kTileW : 0));
  uint64_t* empty = full + p.ST;
  uint64_t* sf_full = empty + p.ST;
  uint64_t* sf_empty = sf_full + kSf<XQ>;
  uint64_t* acc_full = sf_empty + kSf<XQ>;
  uint64_t* acc_free = acc_full + 2;  // one of each per accumulator: the products may run two tiles ahead of the epilogue
  uint64_t* drain = acc_free + 2;
  uint64_t* part_full = drain + 1;
  uint64_t* part_free = part_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part_free + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 2);  // [2] the epilogue warps' common decision
  uint32_t* amax = tmem_slot + 4;  // one CTA: [kEpi][2][4][16] token maxima of the quantizing epilogue
  int* tabs = reinterpret_cast<int*>(amax + kEpi<1> * 128);    // grouped: tile_start and row_start

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = (CG == 2 || p.splits > 1) ? (int)cluster_rank() : 0;
  const int csize = CG == 2 ? 2 : p.splits;  // CTAs that share a tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSf<XQ>; ++s) {
      mbar_init(&sf_full[s], XQ ? 1 + 4 * kEpi<CG> : CG);
      mbar_init(&sf_empty[s], 1);
    }
    mbar_init(&acc_full[0], 1);
    mbar_init(&acc_full[1], 1);
    mbar_init(&acc_free[0], 4 * kEpi<CG> * CG);
    mbar_init(&acc_free[1], 4 * kEpi<CG> * CG);
    mbar_init(drain, 1);
    mbar_init(part_full, 4 * kEpi<CG> * p.splits);
    mbar_init(part_free, 4 * kEpi<CG> * p.splits);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.w);
    if (!XQ) prefetch_tensormap(&maps.x);
  }
  if (warp == 1) tmem_alloc_group<CG>(tmem_slot, (unsigned)p.tmem_cols);
  if (p.groups != 0) {
    // The tables come from the kernel before this one, or (plan_ready) from one that it had waited for before it let this
    // one start: then weights are fetched ahead of the wait as in the dense product.
    if (!p.plan_ready) pdl_wait_prior_grids();
    for (int i = threadIdx.x; i <= p.groups; i += (int)blockDim.x) {
      tabs[i] = p.tile_start[i];
      tabs[p.groups + 1 + i] = p.row_start[i];
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (csize > 1) cluster_sync();  // barriers and tensor memory of the other CTAs are ready
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  pdl_launch_dependents();
  const int tiles = p.n_tiles * (p.groups != 0 ? tabs[p.groups] : p.t_tiles);
  const int first_tile = (int)blockIdx.x / csize, tile_step = (int)gridDim.x / csize;
  const int srank = CG == 2 ? 0 : rank;  // this CTA's part of K
  const int kb0 = (int)((long long)p.KB * srank / p.splits), kb1 = (int)((long long)p.KB * (srank + 1) / p.splits);
  const uint32_t sf_tmem = tmem + (uint32_t)(p.acc_off + NA * p.BT);
  const uint32_t sf_cols = (uint32_t)w8_sf_cols(NA, p.BT);
  const bool apart = p.acc_off >= NA * p.BT;  // the two accumulators share no columns

  if (warp == 0) {
    if (lane == 0) {
      int s = 0, loads = 0;   // ring position; loads saturates at ST (how many stages may be in flight)
      unsigned phase = 1;     // parity of the empty[] phase to wait for: the first round finds its stages free
      auto advance = [&]() {
        if (loads < p.ST) ++loads;
        if (++s == p.ST) {
          s = 0;
          phase ^= 1u;
        }
      };
      const uint32_t base = smem_u32(smem);
      // In a pair both CTAs' copies count on the even CTA's barrier, which expects the bytes of both.
      const uint32_t full0 = CG == 2 ? cluster_addr(full, 0) : smem_u32(full);
      auto load_w = [&](const W8Tile& t, int kb, int s) {
        if (CG == 1 || rank == 0) mbar_arrive_expect_tx(&full[s], (unsigned)(CG * stage));
#pragma unroll
        for (int a = 0; a < NA; ++a)
          tma_load_2d_group<CG>(base + s * stage + a * kTileW * kBlkBytes, &maps.w, kb * kBlkBytes, t.w0 + a * p.N,
                                full0 + s * 8);
      };
      auto load_x = [&](const W8Tile& t, int kb, int s) {
        if (XQ) return;
        tma_load_2d_group<CG>(base + s * stage + NA * kTileW * kBlkBytes, &maps.x, kb * kBlkBytes,
                              t.t0 + (CG == 2 ? rank * (p.BT / 2) : 0), full0 + s * 8);
      };
      bool first = true, ok = true;
      for (int tile = first_tile; tile < tiles && ok; tile += tile_step) {
        const W8Tile t = w8_tile<CG>(p, tabs, tile, rank);
        int kb = kb0;
        if (first) {  // weights do not depend on the kernel before this one: the first ring of them goes ahead of the wait
          first = false;
          const int pre = min(p.ST, kb1 - kb0);
          for (int i = 0; i < pre; ++i) load_w(t, kb0 + i, i);
          pdl_wait_prior_grids();
          for (; kb < kb0 + pre; ++kb) {
            load_x(t, kb, s);
            advance();
          }
        }
        for (; kb < kb1; ++kb) {
          if (!mbar_try_wait(&empty[s], phase) && (*abort_flag || !mbar_wait(&empty[s], phase, p.status))) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          load_w(t, kb, s);
          load_x(t, kb, s);
          advance();
        }
      }
      if (*abort_flag) {  // copies that this thread issued land before the CTA ends
        if (CG == 1 || rank == 0) {
          for (; loads > 0; --loads) {
            if (--s < 0) {
              s = p.ST - 1;
              phase ^= 1u;
            }
            mbar_wait(&full[s], phase ^ 1u, p.status);
          }
        } else {  // counted in the other CTA: a millisecond covers any copy
          const unsigned long long t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
        }
      }
      pdl_wait_prior_grids();
    }
    __syncwarp();
  } else if (warp == 1) {
    // Nothing to multiply before x is there; without this the waits below would count the kernel before this one's time.
    pdl_wait_prior_grids();
    if (CG == 1 || rank == 0) {
      int s = 0, cs = 0, ct = 0, done = 0;  // ring stage, scale slots in shared and tensor memory, tiles
      unsigned phase = 0, cphase = 0;
      int filled = 0;                       // chunks so far, up to kSfTmem
      bool ok = true;
      const uint32_t base = smem_u32(smem), sfbase = smem_u32(sf), xbase = smem_u32(xring);
      for (int tile = first_tile; tile < tiles && ok; tile += tile_step, ++done) {
        // The accumulator is free once the epilogue has read the tile that it held last, two tiles ago (a barrier for each);
        // where the two share columns, once it has read those of the tile before this one (the first barrier).
        if (apart ? done > 1 : done > 0) {
          const bool freed = apart ? warp_wait<CG == 2>(&acc_free[done & 1], (unsigned)((done >> 1) - 1) & 1u, p.status, abort_flag)
                                   : warp_wait<CG == 2>(&acc_free[0], (unsigned)(done - 1) & 1u, p.status, abort_flag);
          if (!freed) break;
        }
        tc_fence_after_sync();
        const uint32_t acc = tmem + ((done & 1) ? (uint32_t)p.acc_off : 0u);
        for (int kb = kb0; kb < kb1; ++kb) {
          const uint32_t sfa = sf_tmem + (uint32_t)ct * sf_cols, sfb = sfa + NA * 4;
          if ((kb & 3) == 0 || kb == kb0) {  // the scales of the next 4 k-blocks
            if (!(ok = warp_wait<CG == 2>(&sf_full[cs], cphase, p.status, abort_flag))) break;
            if (kSf<XQ> <= kSfTmem) {
              // a slot of each kind in step: whoever filled this one had waited for the same products
            } else if (filled < kSfTmem) {
              ++filled;
            } else {  // the products that read this tensor-memory slot last are done (kSfTmem chunks ago)
              const int was = (cs + kSf<XQ> - kSfTmem) % kSf<XQ>;
              if (!(ok = warp_wait(&sf_empty[was], was > cs ? cphase ^ 1u : cphase, p.status, abort_flag))) break;
            }
            tc_fence_after_sync();
            if (elect_one()) {
              const uint64_t d = umma_desc_plain(sfbase + cs * slot);
              for (int a = 0; a * 512 < slot; ++a) tmem_cp_32x128<CG>(sfa + a * 4, d + a * 32);
            }
            __syncwarp();
          }
          if (!(ok = warp_wait(&full[s], phase, p.status, abort_flag))) break;
          tc_fence_after_sync();
          const bool last = (kb & 3) == 3 || kb == kb1 - 1;
          if (elect_one()) {
            const uint64_t wa = umma_desc_sw128(base + s * stage);
            const uint64_t xb = umma_desc_sw128(XQ ? xbase + (cs * 4 + (kb & 3)) * (16 * kBlkBytes)
                                                   : base + s * stage + NA * kTileW * kBlkBytes);
            const uint32_t id = umma_idesc_sf(p.idesc, (uint32_t)(kb & 3));
            // descriptors count 16 bytes: + 2 per 32 channels, + 1024 per set of 128 rows
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_mxf8<CG>(acc + (uint32_t)(a * p.BT), wa + a * 1024 + k * 2, xb + k * 2, id, sfa + a * 4, sfb,
                              k > 0 || kb > kb0);
            umma_commit_group<CG>(&empty[s]);
            if (last) umma_commit_group<CG>(&sf_empty[cs]);
            if (kb == kb1 - 1) umma_commit_group<CG>(&acc_full[done & 1]);
          }
          __syncwarp();
          if (++s == p.ST) {
            s = 0;
            phase ^= 1u;
          }
          if (last) {
            ct = ct + 1 == kSfTmem ? 0 : ct + 1;
            if (++cs == kSf<XQ>) {
              cs = 0;
              cphase ^= 1u;
            }
          }
        }
      }
      if (elect_one()) umma_commit_group<CG>(drain);
      __syncwarp();
    }
  } else if (warp < 4) {
    const int which = warp - 2;
    bool ahead = XQ;  // XQ: this warp's first slot is free; for the next ones the products have to run, and they wait for x
    int turn = 0, cs = 0;
    unsigned phase = 1;
    bool ok = true;
    const int c0 = kb0 >> 2, c1 = (kb1 + 3) >> 2;
    for (int tile = first_tile; tile < tiles && ok; tile += tile_step) {
      const W8Tile t = w8_tile<CG>(p, tabs, tile, rank);
      for (int c = c0; c < c1 && kb0 < kb1; ++c) {
        if (turn == which) {
          uint32_t va[NA][4], vb[8];
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = min(t.w0 + a * p.N + j * 32 + lane, p.wtotal - 1);
              va[a][j] = __ldg(p.ws + (size_t)row * p.SW + c);
            }
          // x's scales come from the kernel before this one, the weight's do not.  XQ: the bounded wait below starts behind that
          // kernel as well, or it would count its time.
          if (!ahead) pdl_wait_prior_grids();
          ahead = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            vb[j] = 0;
            if (!XQ && j * 32 < p.BT) vb[j] = p.xs[(size_t)min(t.t0 + j * 32 + lane, p.xrows - 1) * p.SW + c];
          }
          if (!(ok = warp_wait(&sf_empty[cs], phase, p.status, abort_flag))) break;
          // row i of a 512-byte atom: the words of rows i, i + 32, i + 64, i + 96
          uint4* dst = reinterpret_cast<uint4*>(sf + cs * slot);
#pragma unroll
          for (int a = 0; a < NA; ++a) dst[a * 32 + lane] = make_uint4(va[a][0], va[a][1], va[a][2], va[a][3]);
          if (!XQ) dst[NA * 32 + lane] = make_uint4(vb[0], vb[1], vb[2], vb[3]);
          if (p.BT > 128) dst[(NA + 1) * 32 + lane] = make_uint4(vb[4], vb[5], vb[6], vb[7]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) mbar_arrive_cluster(cluster_addr(&sf_full[cs], 0));
            else mbar_arrive(&sf_full[cs]);
          }
        }
        turn ^= 1;
        if (++cs == kSf<XQ>) {
          cs = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    pdl_wait_prior_grids();
    const int q = warp & 3, row = 32 * q + lane;  // tensor-memory lanes 32 q .. 32 q + 31 are this warp's weight rows
    const int wg = (warp - 4) >> 2;
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    constexpr int CW = CG == 2 ? 16 : 4;  // tokens at a time: few where a tile has few, so that the code stays short
    const int chunks = p.BT / CW;
    const int shared = (NA * p.BT - p.acc_off + CW - 1) / CW;  // chunks whose columns the next tile's accumulator takes
    uint32_t* my_amax = amax + wg * 128;
    int done = 0, turn = 0, decisions = 0;
    XqState xq;
    // All epilogue warps take the same way out: one thread reads the flag for all.
    auto all_ok = [&]() {
      named_barrier_sync(1, 128 * kEpi<CG>);
      if (threadIdx.x == 128) stop[decisions & 1] = *abort_flag;
      named_barrier_sync(1, 128 * kEpi<CG>);
      return stop[decisions++ & 1] == 0;
    };
    auto release = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        uint64_t* bar = &acc_free[apart ? done & 1 : 0];
        if (CG == 2) mbar_arrive_cluster(cluster_addr(bar, 0));
        else mbar_arrive(bar);
      }
    };
    for (int tile = first_tile; tile < tiles; tile += tile_step, ++done) {
      const W8Tile t = w8_tile<CG>(p, tabs, tile, rank);
      if constexpr (XQ) {
        auto quantize = [&](auto dt) {
          w8_quantize_x<decltype(dt)::value>(p, t, xring, sf + NA * 512, slot, sf_full, sf_empty, abort_flag, kb0, kb1,
                                             warp - 4, lane, xq);
        };
        if (p.xdt == AWQ_DTYPE_F16) quantize(std::integral_constant<int, AWQ_DTYPE_F16>{});
        else quantize(std::integral_constant<int, AWQ_DTYPE_BF16>{});
      }
      const bool there = warp_wait(&acc_full[done & 1], (unsigned)(done >> 1) & 1u, p.status, abort_flag);
      if (EPI == kW8Store && CG == 1 ? !there : !all_ok()) break;  // one CTA's stores need no other warp
      tc_fence_after_sync();
      const int buf = done & 1;
      const uint32_t acc = tq + (buf ? (uint32_t)p.acc_off : 0u);
      if (p.splits == 1) {
        bool held = true;
        if (!apart && wg >= shared) {
          release();
          held = false;
        }
        for (int i = wg; i < chunks; i += kEpi<CG>) {
          const int c = CW * (buf ? i : chunks - 1 - i);  // the shared columns are the first buffer's last, the second's first
          uint32_t v[CW], u[CW];
          tmem_ld_cols<CW>(acc + (uint32_t)c, v);
          if (NA == 2) tmem_ld_cols<CW>(acc + (uint32_t)(p.BT + c), u);
          tmem_wait_ld();
          if (held && (apart ? i + kEpi<CG> >= chunks : i + kEpi<CG> >= shared)) {
            release();
            held = false;
          }
          if (c >= t.rows) continue;  // uniform: no token of this chunk exists
          float f[CW], g[CW];
          tmem_cols_f32<CW>(v, f);
          if constexpr (EPI == kW8SiluQuant) tmem_cols_f32<CW>(u, g);
          if constexpr (CG == 2) {
            const uint32_t turned = smem_u32(part + wg * (16 * kTileW));
            if constexpr (EPI == kW8SiluQuant) w8_silu_quant_turned(p, t, row, c, f, g, turned, 2 + wg);
            else if ((p.N & 3) == 0) w8_store_turned(p, t, row, c, f, turned, 2 + wg);
            else w8_store<CW>(p, t, row, c, f);
          } else {
            if constexpr (EPI == kW8SiluQuant) w8_silu_quant<CW>(p, t, row, c, f, g, my_amax, turn, 2 + wg);
            else w8_store<CW>(p, t, row, c, f);
          }
        }
        if (held) release();
        continue;
      }
      // ---- split K: each CTA finishes its share of the tokens.  Every CTA puts its parts straight into the shared memory of
      // the CTA that finishes them, which sums them in rank order: part [rank][accumulator][token of the share][row].
      const bool more = tile + tile_step < tiles;
      const int share = p.BT / p.splits;                     // a multiple of 2
      const uint32_t per_share = (65536u + share - 1) / share;  // t / share = t * per_share >> 16 for t < 64
      if (done > 0) warp_wait(part_free, (unsigned)((done - 1) & 1), p.status, abort_flag);
      for (int c = 16 * wg; c < NA * p.BT; c += 16 * kEpi<CG>) {
        const int a = c >= p.BT ? 1 : 0, t0 = c - a * p.BT;  // the accumulator and its first token here
        if (t0 >= t.rows) continue;
        uint32_t v[16];
        tmem_ld_32x32b_x16(acc + (uint32_t)c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (t0 + j < t.rows) {
            const uint32_t owner = (uint32_t)(t0 + j) * per_share >> 16;
            const int place = (rank * NA + a) * share + (t0 + j - (int)owner * share);
            st_cluster_f32(cluster_addr(part + place * kTileW + row, owner), __uint_as_float(v[j]));
          }
        }
      }
      __syncwarp();
      // one lane per CTA of the cluster: each arrival carries a release, and eight in a row would take microseconds
      if (lane < p.splits) mbar_arrive_cluster(cluster_addr(part_full, (uint32_t)lane));
      if (more) release();
      bool joined = warp_wait<true>(part_full, (unsigned)(done & 1), p.status, abort_flag);
      if (EPI == kW8SiluQuant && !(joined = all_ok())) break;  // its warps meet below, the others nowhere
      const int end = joined ? min(share, t.rows - rank * share) : 0;
      for (int c = 2 * wg; c < end; c += 2 * kEpi<CG>) {
        float f[2] = {0.f, 0.f}, g[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (r < p.splits) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              f[j] += part[(r * NA * share + c + j) * kTileW + row];
              if (NA == 2) g[j] += part[((r * NA + 1) * share + c + j) * kTileW + row];
            }
          }
        }
        if constexpr (EPI == kW8Store) w8_store<2>(p, t, row, rank * share + c, f);
        else w8_silu_quant<2>(p, t, row, rank * share + c, f, g, my_amax, turn, 2 + wg);
      }
      __syncwarp();
      if (more && lane < p.splits) mbar_arrive_cluster(cluster_addr(part_free, (uint32_t)lane));
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  // In-flight products finish before tensor memory is released, and no CTA leaves while another one may still reach it.
  if (warp == 1 && *abort_flag) mbar_wait(drain, 0, p.status);
  if (csize > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_group<CG>(tmem, (unsigned)p.tmem_cols);
  }
}

// ------------------------------------------------------------------------------------------ host
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  return fn;
}

// Codes [rows][K] as 128-byte x `box_rows` boxes in the 128-byte swizzle; columns past K and rows past the end read 0.
bool encode_codes(EncodeTiledFn encode, CUtensorMap* map, const uint8_t* p, long long rows, int K, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {(cuuint32_t)kBlkBytes, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI, int CG, bool XQ>
cudaError_t launch_one(const W8Maps& maps, const W8Params& p, int grid, int smem, cudaStream_t st) {
  static bool ready[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(w8a8_kernel<EPI, CG, XQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW8Smem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kW8Threads<CG>);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)(CG == 2 ? 2 : p.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = attr[1].val.clusterDim.x > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, w8a8_kernel<EPI, CG, XQ>, maps, p);
}

}  // namespace

struct W8Shape {
  int bt, cg, splits;  // tokens per tile, CTAs per tile (1 or 2), parts of K
};

// Parts of K for one-CTA tiles that fill less than half of `slots`, each of kPartLeast k-blocks or more.
int split_k(long long tiles, int KB, int slots) {
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= slots && KB >= splits * 2 * kPartLeast) splits *= 2;
  return splits;
}

// The dense product's tile.  Up to 32 tokens one token tile; above, the tile whose waves over the SMs take the least time by
// a count of cycles: per k-block the larger of the products (2 per token), of their issue (300) and of the operands' way from
// L2 (64 bytes a cycle and SM), a tile's start (1000), the joining of a split K (3000), and the last tile's epilogue (30 per token).
W8Shape dense_shape(int M, int N, int KB, int sms) {
  if (M <= kHalfMost) {
    const int bt = (M + 15) / 16 * 16;
    return W8Shape{bt, 1, split_k((N + kTileW - 1) / kTileW, KB, 2 * sms)};
  }
  W8Shape best{256, 2, 1};
  double least = 1e30;
  for (int bt = 48; bt <= 256; bt += 16) {
    for (int cg = bt < kPairLeast ? 1 : 2; cg >= (bt <= kSplitMost ? 1 : 2); --cg) {
      const long long tiles = (long long)((M + bt - 1) / bt) * ((N + kTileW * cg - 1) / (kTileW * cg));
      const int splits = cg == 1 ? split_k(tiles, KB, sms) : 1;
      const double waves = ceil((double)tiles / (sms / (cg * splits)));
      const double block = fmax(fmax(2.0 * bt, 300.0), (kTileW + (double)bt / cg) * kBlkBytes / 64.0);
      const double cost =
          waves * (ceil((double)KB / splits) * block + 1000.0) + 30.0 * bt + (splits > 1 ? 3000.0 : 0.0);
      if (cost < least) {
        least = cost;
        best = W8Shape{bt, cg, splits};
      }
    }
    if (bt >= M) break;
  }
  return best;
}

bool w8a8_quantizes(int tokens) { return tokens <= kXqMost; }

// The token tile of a grouped product.  Rows spread over the groups at random are about `avg` per group, give or take the
// square root; a tile costs its columns, full or not, and about 32 columns' time for its weights.
int w8a8_grouped_bt(long long rows, int groups, int epi) {
  const long long used = rows < groups ? rows : groups;
  const double avg = (double)rows / (double)used, dev = 1.2 * sqrt(avg);
  const int most = epi == kW8SiluQuant ? 128 : 256;
  int best = 16;
  double least = 1e30;
  for (int bt = 16; bt <= most; bt += 16) {
    double tiles = 0.0;
    for (int k = -1; k <= 1; ++k) tiles += ceil(fmax(avg + k * dev, 1.0) / bt) / 3.0;
    const double cost = tiles * (bt + 32);
    if (cost < least) {
      least = cost;
      best = bt;
    }
  }
  return best;
}

awq_status w8a8_launch(const W8Args& a) {
  const EncodeTiledFn encode = encode_fn();
  if (encode == nullptr) return AWQ_ERR_CUDA;
  const int atoms = a.epi == kW8SiluQuant ? 2 : 1;
  W8Params p = {};
  p.ws = reinterpret_cast<const uint32_t*>(a.wsc);
  p.xs = reinterpret_cast<const uint32_t*>(a.xs);
  p.y = a.y;
  p.hc = a.hc;
  p.hs = a.hs;
  p.row_start = a.row_start;
  p.tile_start = a.tile_start;
  p.plan_ready = a.plan_ready;
  p.status = a.status;
  p.xrows = a.xrows;
  p.wrows = a.N * atoms;
  p.N = a.N;
  p.KB = fp8_blocks(a.K);
  p.SW = fp8_scale_cols(a.K) / 4;
  p.SWh = fp8_scale_cols(a.N) / 4;
  p.groups = a.groups;
  p.dt = a.dt;
  const int sms = num_sms();
  const long long wtotal = (long long)p.wrows * (a.groups ? a.groups : 1);
  // upper bound of the token tiles: grouped, each group that has rows adds at most one partly filled tile
  auto token_tiles = [&](int bt) {
    return a.groups ? (long long)a.xrows / bt + (a.xrows < a.groups ? a.xrows : a.groups) : ((long long)a.xrows + bt - 1) / bt;
  };
  W8Shape shape;
  if (a.groups) {
    shape = W8Shape{a.bt, a.bt >= kPairLeast ? 2 : 1, 1};
    const long long single = token_tiles(a.bt) * ((a.N + kTileW - 1) / kTileW);
    if (a.bt <= kSplitMost) {  // few tiles of a long K are split instead of paired
      const int splits = split_k(single, p.KB, a.bt * atoms <= kHalfMost ? 2 * sms : sms);
      if (shape.cg == 1 || splits > 1) shape = W8Shape{a.bt, 1, splits};
    }
  } else {
    shape = dense_shape(a.xrows, a.N, p.KB, sms);
  }
  const int cg = shape.cg;
  p.BT = shape.bt;
  p.splits = shape.splits;
  p.wtotal = (int)wtotal;
  p.n_tiles = (a.N + kTileW * cg - 1) / (kTileW * cg);
  p.t_tiles = (int)token_tiles(p.BT);
  const long long bound = token_tiles(p.BT) * p.n_tiles;
  if (bound > 0x7FFF0000 || wtotal > 0x7FFF0000) return AWQ_ERR_UNSUPPORTED;
  // Few tokens: two CTAs per SM, so that the next kernel's weights are under way while this one ends.
  const bool half = cg == 1 && p.BT * atoms <= kHalfMost;
  const int slots = half ? 2 * sms : sms;
  const bool xq = a.x != nullptr;
  if (xq && (cg != 1 || a.groups || p.BT > kXqMost)) return AWQ_ERR_UNSUPPORTED;
  const int stage = w8_stage(atoms, xq ? 0 : p.BT / cg), slot = w8_sf_slot(atoms, p.BT);
  const int slots_sf = xq ? kSf<true> * (slot + 4 * 16 * kBlkBytes) : kSf<false> * slot;
  int rest;
  for (;; p.splits /= 2) {  // the parts of a split K and the tables of many groups may leave too little for the ring
    const int part = cg == 2 ? kEpi<2> * 16 * kTileW * 4 : p.splits > 1 ? atoms * p.BT * kTileW * 4 : 0;
    rest = 1024 + slots_sf + part + 512 + 64 + kEpi<1> * 512 + (a.groups ? (2 * a.groups + 2) * 4 : 0);
    p.ST = ((half ? kW8HalfSmem : kW8Smem) - rest) / stage;
    if (p.ST > 12) p.ST = 12;
    if (p.ST >= 2 || p.splits == 1) break;
  }
  if (p.ST < 2) return AWQ_ERR_UNSUPPORTED;
  const int sfc = kSfTmem * w8_sf_cols(atoms, p.BT), acc = atoms * p.BT;
  p.acc_off = acc < 512 - sfc - acc ? acc : 512 - sfc - acc;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.acc_off + acc + sfc) p.tmem_cols <<= 1;
  p.idesc = umma_idesc_mxf8(kTileW * cg, p.BT);
  W8Maps maps;
  if (!encode_codes(encode, &maps.w, a.wc, wtotal, a.K, kTileW)) return AWQ_ERR_CUDA;
  if (xq) {
    p.x = a.x;
    p.K = a.K;
    p.xdt = a.xdt;
  } else if (!encode_codes(encode, &maps.x, a.xc, a.xrows, a.K, p.BT / cg)) {
    return AWQ_ERR_CUDA;
  }
  const int csize = cg == 2 ? 2 : p.splits;
  const long long most_units = slots / csize;
  const int grid = (int)(bound < most_units ? bound : most_units) * csize;
  const int smem = rest + p.ST * stage;
  const bool quant = a.epi == kW8SiluQuant;
  const cudaError_t e = xq ? launch_one<kW8Store, 1, true>(maps, p, grid, smem, a.st)
                        : cg == 2 ? (quant ? launch_one<kW8SiluQuant, 2, false>(maps, p, grid, smem, a.st)
                                           : launch_one<kW8Store, 2, false>(maps, p, grid, smem, a.st))
                                  : (quant ? launch_one<kW8SiluQuant, 1, false>(maps, p, grid, smem, a.st)
                                           : launch_one<kW8Store, 1, false>(maps, p, grid, smem, a.st));
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
