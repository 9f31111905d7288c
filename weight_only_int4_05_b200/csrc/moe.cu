// moe.cu -- w8a8_moe: the expert MLP of a sparse layer on 8-bit weights, from the router's choice to the output.
//
//   y_m = sum_j w_mj  Wd[e] Q(silu(a) b),   a | b = Wgu[e] Q(x_m),   e = ids_mj,
// with Q the 8-bit quantizer (fp8.cuh).  A token's copies are sorted by expert (stable, so the order does not depend on
// timing), quantized straight into that order, and met with the experts' weights by the grouped product of w8a8.cu; its
// first pass ends in silu(gate) up quantized again, its second in 32-bit rows that the combine sums slot by slot.
// Kernels: up to 1024 copies plan_kernel (ranks, tables and the quantized rows in one launch); more, rank_kernel (rank of
// each copy within its expert, by chunks of 1024), place_kernel (the tables of the grouped product) and scatter_kernel (quantizes
// into the sorted order); then 2 x w8a8_kernel and combine_kernel.
// Measured (B200): one token, top 2 of 8 experts 4096/14336: 70 us, 5.1 TB/s of the two experts' bytes (54 us at the copy rate).
// 2048 tokens, top 6 of 64 experts 4096/1024: 283 - 336 us; alone the kernels take rank 5, place 6, scatter 13.5, gate|up 114,
// down 95 - 101, combine 33, the products at 82 and 73 % of the copy rate: the 32-bit rows of the down projection (201 MB each way)
// cost about 60 of them, which rounding the rows to 16 bits would halve at 1.4 times the output's rounding error.
#include "fp8.cuh"
#include "w8a8.cuh"

namespace awq {

namespace {

constexpr int kChunk = 1024;  // copies (token, slot) per block of rank_kernel: one per thread

struct Plan {  // device tables of one call, in the workspace
  int* rank;        // [A] rank within (chunk, expert), -1 without an expert
  int* pos;         // [A] row of the sorted order, -1 without an expert
  int* hist;        // [chunks][E] counts, then the copies of earlier chunks
  int* row_start;   // [E + 1]
  int* tiles_gu;    // [E + 1] token tiles before each expert, gate|up
  int* tiles_d;     // [E + 1] the same, down
};

struct Layout {
  size_t xc, xs, hc, hs, d, rank, pos, hist, row_start, tiles_gu, tiles_d, total;
};

Layout layout(int M, int E, int topk, int K, int I, int N) {
  const size_t A = (size_t)M * topk, chunks = (A + kChunk - 1) / kChunk;
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  l.xc = take(A * K);
  l.xs = take(A * fp8_scale_cols(K));
  l.hc = take(A * I);
  l.hs = take(A * fp8_scale_cols(I));
  l.d = take(A * N * sizeof(float));
  l.rank = take(A * sizeof(int));
  l.pos = take(A * sizeof(int));
  l.hist = take(chunks * E * sizeof(int));
  l.row_start = take((size_t)(E + 1) * sizeof(int));
  l.tiles_gu = take((size_t)(E + 1) * sizeof(int));
  l.tiles_d = take((size_t)(E + 1) * sizeof(int));
  l.total = at;
  return l;
}

// Exclusive sums of the experts' counts (count [E] in shared memory, replaced by each expert's first row) and of their
// token tiles, written to the tables where `write`.  1024 threads, E <= 1024.
__device__ __forceinline__ void place_tables(const Plan& t, int E, int bt_gu, int bt_d, int* count, bool write) {
  __shared__ int warp_sum[3][32];
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  const int n = e < E ? count[e] : 0;
  int v[3] = {n, (n + bt_gu - 1) / bt_gu, (n + bt_d - 1) / bt_d};
  int* out[3] = {t.row_start, t.tiles_gu, t.tiles_d};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int s = v[i];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += o;
    }
    if (lane == 31) warp_sum[i][warp] = s;
    v[i] = s;  // inclusive within the warp
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[i][w];
    if (write && e < E) out[i][e + 1] = before + v[i];
    if (write && e == 0) out[i][0] = 0;
    if (i == 0 && e < E) count[e] = before + v[i] - n;
  }
  __syncthreads();
}

// Stable rank of this thread's copy (expert e, -1: none) among the copies of its expert in the chunk: lanes of one warp by
// match, warps by a scan of their counts in wcnt [32][E]; total [E] gets the chunk's counts.
__device__ __forceinline__ int rank_chunk(int e, int E, uint16_t* wcnt, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 32 * E; i += kChunk) wcnt[i] = 0;
  __syncthreads();
  const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e);
  const int below = __popc(peers & ((1u << lane) - 1u));
  if (e >= 0 && below == 0) wcnt[warp * E + e] = (uint16_t)__popc(peers);
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kChunk) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      const int v = wcnt[w * E + i];
      wcnt[w * E + i] = (uint16_t)sum;
      sum += v;
    }
    total[i] = sum;
  }
  __syncthreads();
  return e < 0 ? -1 : wcnt[warp * E + e] + below;
}

// 512 columns of one token (from column 512 w on) quantized by a warp: two pieces of 8 codes per lane, and lane 0's word of
// scales (the layout of fp8_quantize_kernel).
template <int DT>
__device__ __forceinline__ uint32_t quantize_512(const uint16_t* x, int K, int w, int lane, uint2 (&c)[2]) {
  uint4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = w * 512 + h * 256 + lane * 8;
    v[h] = make_uint4(0u, 0u, 0u, 0u);
    if (k < K) v[h] = ldg_stream(x + k);
  }
  uint32_t word = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
    float f[8], m = 0.f;
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
    c[h].x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
    c[h].y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
    word |= (b | (__shfl_sync(0xFFFFFFFFu, b, 16) << 8)) << (16 * h);  // lane 0's word: the blocks of lanes 0 and 16
  }
  return word;
}

// Writes a token's 512 columns to the sorted rows of its copies; lane j holds copy j's row (-1: none).
__device__ __forceinline__ void write_copies(int to, int topk, int K, int SW, int w, int lane, const uint2 (&c)[2],
                                             uint32_t word, uint8_t* codes, uint32_t* scales) {
  for (int j = 0; j < topk; ++j) {
    const int r = __shfl_sync(0xFFFFFFFFu, to, j);
    if (r < 0) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = w * 512 + h * 256 + lane * 8;
      if (k < K) *reinterpret_cast<uint2*>(codes + (size_t)r * K + k) = c[h];
    }
    if (lane == 0) scales[(size_t)r * SW + w] = word;
  }
}

}  // namespace

// Up to 1024 copies: every block ranks all of them (a few microseconds, less than a launch between two kernels) and then
// quantizes its share of the tokens; block 0 writes the tables.
template <int DT>
__global__ void __launch_bounds__(kChunk) plan_kernel(const uint16_t* x, const int32_t* ids, int A, int E, int M, int topk,
                                                      int K, int SW, Plan t, int bt_gu, int bt_d, uint8_t* codes,
                                                      uint32_t* scales) {
  extern __shared__ uint16_t wcnt[];  // [32][E]
  __shared__ int first_row[kChunk], row_of[kChunk];
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, a = threadIdx.x;
  int e = a < A ? ids[a] : -1;
  if (e < 0 || e >= E) e = -1;
  const int rank = rank_chunk(e, E, wcnt, first_row);
  place_tables(t, E, bt_gu, bt_d, first_row, blockIdx.x == 0);
  row_of[a] = e < 0 ? -1 : first_row[e] + rank;
  if (blockIdx.x == 0 && a < A) t.pos[a] = row_of[a];
  __syncthreads();
  const int items = M * SW;
  for (int it = blockIdx.x * 32 + warp; it < items; it += gridDim.x * 32) {
    const int row = it / SW, w = it - row * SW;
    uint2 c[2];
    const uint32_t word = quantize_512<DT>(x + (size_t)row * K, K, w, lane, c);
    write_copies(lane < topk ? row_of[row * topk + lane] : -1, topk, K, SW, w, lane, c, word, codes, scales);
  }
}

__global__ void __launch_bounds__(kChunk) rank_kernel(const int32_t* ids, int A, int E, Plan t) {
  extern __shared__ uint16_t wcnt[];  // [32][E]
  __shared__ int total[kChunk];
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int a = blockIdx.x * kChunk + threadIdx.x;
  int e = a < A ? ids[a] : -1;
  if (e < 0 || e >= E) e = -1;
  const int rank = rank_chunk(e, E, wcnt, total);
  if (a < A) t.rank[a] = rank;
  for (int i = threadIdx.x; i < E; i += kChunk) t.hist[(size_t)blockIdx.x * E + i] = total[i];
}

// Exclusive sums over the chunks of each expert (a warp per expert, a lane per chunk), then the tables.
__global__ void __launch_bounds__(1024) place_kernel(Plan t, int E, int chunks, int bt_gu, int bt_d) {
  __shared__ int count[1024];
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int x = warp; x < E; x += 32) {
    int total = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const int c = c0 + lane;
      const int v = c < chunks ? t.hist[(size_t)c * E + x] : 0;
      int s = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += o;
      }
      if (c < chunks) t.hist[(size_t)c * E + x] = total + s - v;
      total += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) count[x] = total;
  }
  __syncthreads();
  place_tables(t, E, bt_gu, bt_d, count, true);
}

// Quantizes each token once and writes it to the sorted rows of all its copies, one warp per 512 columns of a token.
template <int DT>
__global__ void __launch_bounds__(256) scatter_kernel(const uint16_t* x, const int32_t* ids, int M, int E, int topk, int K,
                                                      int SW, Plan t, uint8_t* codes, uint32_t* scales) {
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const long long items = (long long)M * SW;
  const long long step = (long long)gridDim.x * (blockDim.x >> 5);
  for (long long it = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += step) {
    const long long row = it / SW;
    const int w = (int)(it - row * SW);
    int to = -1;  // lane j: the row of the token's copy j
    if (lane < topk) {
      const long long a = row * topk + lane;
      const int rank = t.rank[a];
      if (rank >= 0) {
        const int e = ids[a];
        to = t.row_start[e] + t.hist[(size_t)(a / kChunk) * E + e] + rank;
      }
      if (w == 0) t.pos[a] = to;
    }
    uint2 c[2];
    const uint32_t word = quantize_512<DT>(x + row * K, K, w, lane, c);
    write_copies(to, topk, K, SW, w, lane, c, word, codes, scales);
  }
}

// y_m = round(sum_j w_mj d[pos_mj]), slots in order, 32 bits until the end.  One thread per 4 columns of a token; the rows
// of 4 slots are fetched together, since a fetch after each slot's place would wait for memory twice per slot.
template <bool WIDE>
__global__ void __launch_bounds__(256) combine_kernel(const float* d, const int* pos, const float* weights, int M, int topk,
                                                      int N, int dt, uint16_t* y) {
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int cols = (N + 3) / 4;
  const long long items = (long long)M * cols;
  for (long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x; it < items;
       it += (long long)gridDim.x * blockDim.x) {
    const int m = (int)(it / cols);
    const int n = (int)(it - (long long)m * cols) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < topk; j0 += 4) {
      int r[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = j0 + j < topk ? pos[(size_t)m * topk + j0 + j] : -1;
        w[j] = j0 + j < topk ? weights[(size_t)m * topk + j0 + j] : 0.f;
      }
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r[j] < 0) continue;
        const float* src = d + (size_t)r[j] * N + n;
        if (WIDE) v[j] = *reinterpret_cast<const float4*>(src);
        else v[j] = make_float4(src[0], n + 1 < N ? src[1] : 0.f, n + 2 < N ? src[2] : 0.f, n + 3 < N ? src[3] : 0.f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r[j] < 0) continue;  // a weight of an empty slot may be anything
        s.x = fmaf(w[j], v[j].x, s.x);
        s.y = fmaf(w[j], v[j].y, s.y);
        s.z = fmaf(w[j], v[j].z, s.z);
        s.w = fmaf(w[j], v[j].w, s.w);
      }
    }
    uint16_t* o = y + (size_t)m * N + n;
    const float f[4] = {s.x, s.y, s.z, s.w};
    if (WIDE) {
      uint2 v;
      v.x = f32_to_16(f[0], dt) | ((uint32_t)f32_to_16(f[1], dt) << 16);
      v.y = f32_to_16(f[2], dt) | ((uint32_t)f32_to_16(f[3], dt) << 16);
      *reinterpret_cast<uint2*>(o) = v;
    } else {
      for (int i = 0; i < 4 && n + i < N; ++i) o[i] = f32_to_16(f[i], dt);
    }
  }
}

size_t moe_workspace_bytes(int M, int E, int topk, int K, int I, int N) { return layout(M, E, topk, K, I, N).total; }

awq_status moe_launch(const MoeArgs& a) {
  const Layout l = layout(a.M, a.E, a.topk, a.K, a.I, a.N);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const int A = a.M * a.topk, chunks = (A + kChunk - 1) / kChunk;
  const Plan t{reinterpret_cast<int*>(ws + l.rank),      reinterpret_cast<int*>(ws + l.pos),
               reinterpret_cast<int*>(ws + l.hist),      reinterpret_cast<int*>(ws + l.row_start),
               reinterpret_cast<int*>(ws + l.tiles_gu), reinterpret_cast<int*>(ws + l.tiles_d)};
  const int bt_gu = w8a8_grouped_bt(A, a.E, kW8SiluQuant), bt_d = w8a8_grouped_bt(A, a.E, kW8Store);
  const size_t cnt = (size_t)32 * a.E * sizeof(uint16_t);  // at most 64 KB
  auto plan = a.dt == AWQ_DTYPE_F16 ? plan_kernel<AWQ_DTYPE_F16> : plan_kernel<AWQ_DTYPE_BF16>;
  if (cnt > 32 * 1024 &&  // with the static tables the default limit is near
      (cudaFuncSetAttribute(rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess ||
       cudaFuncSetAttribute(plan, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess))
    return AWQ_ERR_CUDA;
  const int SW = fp8_scale_cols(a.K) / 4, sms = num_sms();
  const long long cap = (long long)sms * 8;
  const long long warps = (long long)a.M * SW;
  long long blocks = (warps + 31) / 32;
  uint32_t* xs = reinterpret_cast<uint32_t*>(ws + l.xs);
  cudaError_t e;
  if (chunks == 1) {
    e = launch_pdl(plan, dim3((unsigned)(blocks < sms ? blocks : sms)), dim3(kChunk), cnt, a.st, a.x, a.ids, A, a.E, a.M,
                   a.topk, a.K, SW, t, bt_gu, bt_d, ws + l.xc, xs);
  } else {
    e = launch_pdl(rank_kernel, dim3((unsigned)chunks), dim3(kChunk), cnt, a.st, a.ids, A, a.E, t);
    if (e == cudaSuccess)
      e = launch_pdl(place_kernel, dim3(1), dim3(1024), 0, a.st, t, a.E, chunks, bt_gu, bt_d);
    auto scatter = a.dt == AWQ_DTYPE_F16 ? scatter_kernel<AWQ_DTYPE_F16> : scatter_kernel<AWQ_DTYPE_BF16>;
    blocks = (warps + 7) / 8;
    if (e == cudaSuccess)
      e = launch_pdl(scatter, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, a.st, a.x, a.ids, a.M, a.E,
                     a.topk, a.K, SW, t, ws + l.xc, xs);
  }
  if (e != cudaSuccess) return AWQ_ERR_CUDA;
  W8Args g;
  g.groups = a.E;
  g.row_start = t.row_start;
  g.xrows = A;
  g.status = a.status;
  g.st = a.st;
  W8Args up = g;
  up.xc = ws + l.xc;
  up.xs = ws + l.xs;
  up.wc = a.guc;
  up.wsc = a.gus;
  up.N = a.I;
  up.K = a.K;
  up.tile_start = t.tiles_gu;
  up.bt = bt_gu;
  up.epi = kW8SiluQuant;
  up.hc = ws + l.hc;
  up.hs = ws + l.hs;
  awq_status st = w8a8_launch(up);
  if (st != AWQ_OK) return st;
  W8Args down = g;
  down.xc = ws + l.hc;
  down.xs = ws + l.hs;
  down.wc = a.dc;
  down.wsc = a.ds;
  down.N = a.N;
  down.K = a.I;
  down.tile_start = t.tiles_d;
  down.bt = bt_d;
  down.y = ws + l.d;
  down.dt = AWQ_DTYPE_F32;
  down.plan_ready = true;  // the first product waits for the plan before it lets the second start
  st = w8a8_launch(down);
  if (st != AWQ_OK) return st;
  blocks = ((long long)a.M * ((a.N + 3) / 4) + 255) / 256;
  auto combine = a.N % 4 == 0 ? combine_kernel<true> : combine_kernel<false>;
  e = launch_pdl(combine, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, a.st,
                 reinterpret_cast<const float*>(ws + l.d), static_cast<const int*>(t.pos), a.weights, a.M, a.topk, a.N,
                 a.dt, a.y);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
