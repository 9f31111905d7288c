// w8a8.cu -- the product of two 8-bit block-scaled matrices on the tcgen05 tensor cores.
//
// y^T tile [128 weight rows][BT tokens] = sum over blocks of 128 channels of (C_w T_w) . (C_x T_x)^T, with e4m3 codes C and
// power-of-two scales T.  The scales go to tensor memory beside the accumulator and the tensor cores apply them
// (kind::mxf8f6f4.block_scale): one scale byte serves the four 32-channel steps of its block, so a block of 128 costs
// the same as the format's native 32 and no partial sum leaves tensor memory.  Weights are the A operand (128 rows of
// N), tokens the B operand, so a few tokens still fill the instruction's height.
//
// Per CTA (8 warps), persistent over output tiles, k-blocks of 128 channels through an ST-stage ring:
//   warp 0      producer: TMA copies of the weight rows and of the tokens (128-byte swizzle) onto full[s].
//   warp 1      MMA: per k-block 4 x tcgen05.mma (32 channels each); every 4th k-block first copies the next scale words
//               from shared to tensor memory (tcgen05.cp, two slots).
//   warps 2, 3  scales: one 32-bit word per row holds the scales of 4 k-blocks; each warp fills one of two slots.
//   warps 4..7  epilogue: tensor memory -> registers -> y, or h = silu(gate) up quantized again.
// Every mbarrier wait is bounded; a timeout is recorded in the status word, the CTA drains its copies and MMAs, frees
// its tensor memory and exits.
#include "fp8.cuh"
#include "w8a8.cuh"

namespace awq {

namespace {

constexpr int kTileW = 128;        // weight rows per accumulator
constexpr int kBlkBytes = 128;     // bytes of K per k-block: one swizzle row, one scale block
constexpr int kW8Threads = 256;
constexpr int kW8Smem = 232448;    // opt-in dynamic shared memory per block on sm_100
constexpr int kMaxGroups = 1024;

struct W8Params {
  const uint32_t* ws;  // scale words of w and x, SW per row
  const uint32_t* xs;
  void* y;
  uint8_t* hc;
  uint8_t* hs;
  const int* row_start;
  const int* tile_start;
  unsigned* status;
  int xrows, wrows, wtotal;  // rows of x, weight rows per group, weight rows in all
  int N, K, KB, SW, SWh;
  int BT, ST, tmem_cols, groups, n_tiles, t_tiles, dt;
  uint32_t idesc;
};

struct W8Tile {
  int w0, n0, t0, rows;  // first weight row (in the stack of all groups), first output, first token row, valid token rows
};

template <int EPI>
constexpr int kAtomsA = EPI == kW8SiluQuant ? 2 : 1;  // accumulators (weight row sets) per tile

__host__ __device__ constexpr int w8_stage(int atoms, int BT) { return (atoms * kTileW + BT) * kBlkBytes; }
__host__ __device__ constexpr int w8_sf_slot(int atoms, int BT) { return (atoms + (BT + 127) / 128) * 512; }

// Tile number -> place.  Dense: token tiles fastest, so the tiles in flight share weight rows.  Grouped: group by group,
// token tiles fastest within a weight tile; tabs = [tile_start | row_start] in shared memory.
__device__ __forceinline__ W8Tile w8_tile(const W8Params& p, const int* tabs, int tile) {
  W8Tile r;
  if (p.groups == 0) {
    const int n = tile / p.t_tiles, t = tile - n * p.t_tiles;
    r.n0 = n * kTileW;
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
  r.n0 = n * kTileW;
  r.w0 = lo * p.wrows + r.n0;
  r.t0 = rows[lo] + t * p.BT;
  r.rows = min(p.BT, rows[lo + 1] - r.t0);
  return r;
}

struct W8Maps {
  CUtensorMap w, x;
};

__device__ __forceinline__ float w8_silu(float a) { return a / (1.0f + expf(-a)); }

}  // namespace

template <int EPI>
__global__ void __launch_bounds__(kW8Threads, 1) w8a8_kernel(const __grid_constant__ W8Maps maps, const W8Params p) {
  constexpr int NA = kAtomsA<EPI>;
  extern __shared__ uint8_t w8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(w8_smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage = w8_stage(NA, p.BT), slot = w8_sf_slot(NA, p.BT);
  uint8_t* sf = smem + (size_t)p.ST * stage;
  uint64_t* full = reinterpret_cast<uint64_t*>(sf + 2 * slot);
  uint64_t* empty = full + p.ST;
  uint64_t* sf_full = empty + p.ST;
  uint64_t* sf_empty = sf_full + 2;
  uint64_t* acc_full = sf_empty + 2;
  uint64_t* acc_free = acc_full + 1;
  uint64_t* drain = acc_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 2);  // [2] the epilogue warps' common decision
  uint32_t* amax = tmem_slot + 4;                    // [2][4][16] row maxima of the quantizing epilogue
  int* tabs = reinterpret_cast<int*>(amax + 128);    // grouped: tile_start and row_start

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, (unsigned)p.tmem_cols);
    tmem_relinquish();
  }
  if (p.groups != 0) {
    pdl_wait_prior_grids();
    for (int i = threadIdx.x; i <= p.groups; i += kW8Threads) {
      tabs[i] = p.tile_start[i];
      tabs[p.groups + 1 + i] = p.row_start[i];
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  const int tiles = p.n_tiles * (p.groups != 0 ? tabs[p.groups] : p.t_tiles);
  const uint32_t sf_tmem = tmem + (uint32_t)(NA * p.BT);
  const uint32_t sf_cols = (uint32_t)(NA * 4 + (p.BT + 127) / 128 * 4);

  if (warp == 0) {
    if (lane == 0) {
      const unsigned tx = (unsigned)stage;
      long long it = 0;
      bool first = true;
      auto load_w = [&](const W8Tile& t, int kb, int s) {
        uint8_t* st = smem + (size_t)s * stage;
        mbar_arrive_expect_tx(&full[s], tx);
#pragma unroll
        for (int a = 0; a < NA; ++a)
          tma_load_2d(st + a * kTileW * kBlkBytes, &maps.w, kb * kBlkBytes, t.w0 + a * p.N, &full[s]);
      };
      auto load_x = [&](const W8Tile& t, int kb, int s) {
        tma_load_2d(smem + (size_t)s * stage + NA * kTileW * kBlkBytes, &maps.x, kb * kBlkBytes, t.t0, &full[s]);
      };
      for (int tile = blockIdx.x; tile < tiles && !*abort_flag; tile += gridDim.x) {
        const W8Tile t = w8_tile(p, tabs, tile);
        int kb = 0;
        if (first) {  // weights do not depend on the kernel before this one: the first ring of them goes ahead of the wait
          first = false;
          const int pre = min(p.ST, p.KB);
          for (; kb < pre; ++kb) load_w(t, kb, kb);
          pdl_wait_prior_grids();
          for (kb = 0; kb < pre; ++kb) load_x(t, kb, kb);
          it = pre;
        }
        for (; kb < p.KB; ++kb, ++it) {
          const int s = (int)(it % p.ST);
          if (it >= p.ST && (*abort_flag || !mbar_wait(&empty[s], (unsigned)((it / p.ST - 1) & 1), p.status))) {
            *abort_flag = 1;
            break;
          }
          load_w(t, kb, s);
          load_x(t, kb, s);
        }
      }
      if (*abort_flag) {  // every copy that this thread issued lands before the CTA ends
        for (long long i = it > p.ST ? it - p.ST : 0; i < it; ++i)
          mbar_wait(&full[i % p.ST], (unsigned)((i / p.ST) & 1), p.status);
      }
      pdl_wait_prior_grids();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      long long it = 0;
      int cc = 0, done = 0;
      for (int tile = blockIdx.x; tile < tiles && !*abort_flag; tile += gridDim.x, ++done) {
        if (done > 0 && !mbar_wait(acc_free, (unsigned)((done - 1) & 1), p.status)) {
          *abort_flag = 1;
          break;
        }
        tc_fence_after_sync();
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const int s = (int)(it % p.ST), c = cc & 1;
          const uint32_t sfa = sf_tmem + (uint32_t)c * sf_cols, sfb = sfa + NA * 4;
          if ((kb & 3) == 0) {  // the scales of the next 4 k-blocks
            if (*abort_flag || !mbar_wait(&sf_full[c], (unsigned)((cc >> 1) & 1), p.status)) {
              *abort_flag = 1;
              break;
            }
            tc_fence_after_sync();
            for (int a = 0; a * 512 < slot; ++a)
              tmem_cp_32x128(sfa + a * 4, umma_desc_plain(smem_u32(sf + (size_t)c * slot + a * 512)));
          }
          if (*abort_flag || !mbar_wait(&full[s], (unsigned)((it / p.ST) & 1), p.status)) {
            *abort_flag = 1;
            break;
          }
          tc_fence_after_sync();
          const uint32_t wa = smem_u32(smem + (size_t)s * stage), xb = wa + NA * kTileW * kBlkBytes;
          const uint32_t id = umma_idesc_sf(p.idesc, (uint32_t)(kb & 3));
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_mxf8(tmem + (uint32_t)(a * p.BT), umma_desc_sw128(wa + a * kTileW * kBlkBytes + k * 32),
                        umma_desc_sw128(xb + k * 32), id, sfa + a * 4, sfb, (kb | k) != 0);
          umma_commit(&empty[s]);
          if ((kb & 3) == 3 || kb == p.KB - 1) {
            umma_commit(&sf_empty[c]);
            ++cc;
          }
        }
        if (*abort_flag) break;
        umma_commit(acc_full);
      }
      umma_commit(drain);
    }
  } else if (warp < 4) {
    const int which = warp - 2;
    int cc = 0;
    pdl_wait_prior_grids();
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
      const W8Tile t = w8_tile(p, tabs, tile);
      for (int c = 0; c * 4 < p.KB; ++c, ++cc) {
        if ((cc & 1) != which) continue;
        uint32_t va[NA][4], vb[8];
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = min(t.w0 + a * p.N + j * 32 + lane, p.wtotal - 1);
            va[a][j] = __ldg(p.ws + (size_t)row * p.SW + c);
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          vb[j] = 0;
          if (j * 32 < p.BT) vb[j] = p.xs[(size_t)min(t.t0 + j * 32 + lane, p.xrows - 1) * p.SW + c];
        }
        if (cc >= 2 && (*abort_flag || !mbar_wait_backoff(&sf_empty[which], (unsigned)(((cc >> 1) - 1) & 1), p.status)))
          *abort_flag = 1;
        __syncwarp();
        if (__shfl_sync(0xFFFFFFFFu, *abort_flag, 0)) {  // one lane reads the flag for all
          ok = false;
          break;
        }
        // row i of a 512-byte atom: the words of rows i, i + 32, i + 64, i + 96
        uint4* dst = reinterpret_cast<uint4*>(sf + (size_t)which * slot);
#pragma unroll
        for (int a = 0; a < NA; ++a) dst[a * 32 + lane] = make_uint4(va[a][0], va[a][1], va[a][2], va[a][3]);
        dst[NA * 32 + lane] = make_uint4(vb[0], vb[1], vb[2], vb[3]);
        if (p.BT > 128) dst[(NA + 1) * 32 + lane] = make_uint4(vb[4], vb[5], vb[6], vb[7]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[which]);
      }
    }
  } else {
    pdl_wait_prior_grids();
    const int q = warp & 3, row = 32 * q + lane;  // tensor-memory lanes 32 q .. 32 q + 31 are this warp's weight rows
    const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
    int done = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++done) {
      const W8Tile t = w8_tile(p, tabs, tile);
      if (*abort_flag || !mbar_wait(acc_full, (unsigned)(done & 1), p.status)) *abort_flag = 1;
      named_barrier_sync(1, 128);  // the four warps take the same way out: one thread reads the flag for all
      if (threadIdx.x == 128) stop[done & 1] = *abort_flag;
      named_barrier_sync(1, 128);
      if (stop[done & 1]) break;
      tc_fence_after_sync();
      const int n = t.n0 + row;
      for (int c0 = 0; c0 < p.BT; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tq + (uint32_t)c0, v);
        if constexpr (EPI == kW8Store) {
          tmem_wait_ld();
          if (n < p.N) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c0 + i < t.rows) {
                const size_t at = (size_t)(t.t0 + c0 + i) * p.N + n;
                const float f = __uint_as_float(v[i]);
                if (p.dt == AWQ_DTYPE_F32) static_cast<float*>(p.y)[at] = f;
                else static_cast<uint16_t*>(p.y)[at] = f32_to_16(f, p.dt);
              }
            }
          }
        } else {
          uint32_t u[16];
          tmem_ld_32x32b_x16(tq + (uint32_t)(p.BT + c0), u);
          tmem_wait_ld();
          const int buf = (c0 >> 4) & 1;
          float h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            h[i] = n < p.N ? w8_silu(__uint_as_float(v[i])) * __uint_as_float(u[i]) : 0.f;
            const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h[i])));
            if (lane == i) amax[(buf * 4 + q) * 16 + i] = m;
          }
          named_barrier_sync(1, 128);  // two buffers: the next chunk's maxima do not meet this chunk's readers
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t* am = amax + buf * 64 + i;
            const uint32_t b = fp8_scale_byte(max(max(am[0], am[16]), max(am[32], am[48])));
            if (c0 + i < t.rows) {
              const size_t r = (size_t)(t.t0 + c0 + i);
              if (n < p.N) p.hc[r * p.N + n] = (uint8_t)e4m3x2(h[i] * fp8_inv_scale(b), 0.f);
              if (row == 0) p.hs[r * (p.SWh * 4) + t.n0 / kFp8Block] = (uint8_t)b;
            }
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    if (*abort_flag) mbar_wait(drain, 0, p.status);  // MMAs in flight finish before tensor memory is released
    tc_fence_after_sync();
    tmem_dealloc(tmem, (unsigned)p.tmem_cols);
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

template <int EPI>
cudaError_t launch_one(const W8Maps& maps, const W8Params& p, int grid, int smem, cudaStream_t st) {
  static bool ready[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(w8a8_kernel<EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW8Smem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  return launch_pdl(w8a8_kernel<EPI>, dim3((unsigned)grid), dim3(kW8Threads), (size_t)smem, st, maps, p);
}

}  // namespace

int w8a8_grouped_bt(long long rows, int groups, int epi) {
  const long long used = rows < groups ? rows : groups;
  const long long avg = (rows + used - 1) / used;
  const int most = epi == kW8SiluQuant ? 128 : 256;
  int bt = 16;
  while (bt < avg && bt < most) bt <<= 1;
  return bt;
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
  p.status = a.status;
  p.xrows = a.xrows;
  p.wrows = a.N * atoms;
  p.N = a.N;
  p.K = a.K;
  p.KB = fp8_blocks(a.K);
  p.SW = fp8_scale_cols(a.K) / 4;
  p.SWh = fp8_scale_cols(a.N) / 4;
  p.groups = a.groups;
  p.dt = a.dt;
  const int most = a.epi == kW8SiluQuant ? 128 : 256;
  p.BT = a.groups ? a.bt : a.xrows >= most ? most : (a.xrows + 15) / 16 * 16;
  const long long wtotal = (long long)p.wrows * (a.groups ? a.groups : 1);
  p.wtotal = (int)wtotal;
  p.n_tiles = (a.N + kTileW - 1) / kTileW;
  p.t_tiles = (a.xrows + p.BT - 1) / p.BT;
  // upper bound of the tiles: grouped, each group that has rows adds at most one partly filled token tile
  const long long tt = a.groups ? (a.xrows / p.BT + (a.xrows < a.groups ? a.xrows : a.groups)) : p.t_tiles;
  const long long bound = tt * p.n_tiles;
  if (bound > 0x7FFFFFFF || wtotal > 0x7FFFFFFF) return AWQ_ERR_UNSUPPORTED;
  const int stage = w8_stage(atoms, p.BT), slot = w8_sf_slot(atoms, p.BT);
  const int rest = 1024 + 2 * slot + 2 * 16 * 8 + 64 + 512 + 64 + (a.groups ? (2 * a.groups + 2) * 4 : 0);
  p.ST = (kW8Smem - rest) / stage;
  if (p.ST > 12) p.ST = 12;
  const int cols = atoms * p.BT + 2 * (atoms * 4 + (p.BT + 127) / 128 * 4);
  p.tmem_cols = 32;
  while (p.tmem_cols < cols) p.tmem_cols <<= 1;
  if (p.ST < 2 || p.tmem_cols > 512) return AWQ_ERR_UNSUPPORTED;
  p.idesc = umma_idesc_mxf8(kTileW, p.BT);
  W8Maps maps;
  if (!encode_codes(encode, &maps.w, a.wc, wtotal, a.K, kTileW) ||
      !encode_codes(encode, &maps.x, a.xc, a.xrows, a.K, p.BT))
    return AWQ_ERR_CUDA;
  const int sms = num_sms();
  const int grid = bound < sms ? (int)bound : sms;
  const int smem = rest + p.ST * stage;
  const cudaError_t e = a.epi == kW8SiluQuant ? launch_one<kW8SiluQuant>(maps, p, grid, smem, a.st)
                                              : launch_one<kW8Store>(maps, p, grid, smem, a.st);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
