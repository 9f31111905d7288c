// moe.cu -- w8a8_moe: the expert MLP of a sparse layer on 8-bit weights, from the router's choice to the output.
//
//   y_m = sum_j w_mj  Wd[e] Q(silu(a) b),   a | b = Wgu[e] Q(x_m),   e = ids_mj,
// with Q the 8-bit quantizer (fp8.cuh).  A token's copies are sorted by expert (stable, so the order does not depend on
// timing), quantized straight into that order, and met with the experts' weights by the grouped product of w8a8.cu; its
// first pass ends in silu(gate) up quantized again, its second in 32-bit rows that the combine sums slot by slot.
// Kernels: rank_kernel (rank of each copy within its expert, by chunks of 1024), place_kernel (the tables of the grouped
// product; one launch with rank_kernel when there is one chunk), scatter_kernel, 2 x w8a8_kernel, combine_kernel.
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

// Exclusive sums over the chunks of each expert, over the experts, and of their token tiles.  1024 threads, E <= 1024.
__device__ __forceinline__ void place_tables(const Plan& t, int E, int chunks, int bt_gu, int bt_d) {
  __shared__ int warp_sum[3][32];
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  int count = 0;
  if (e < E)
    for (int c = 0; c < chunks; ++c) {
      const int v = t.hist[(size_t)c * E + e];
      t.hist[(size_t)c * E + e] = count;
      count += v;
    }
  int v[3] = {count, (count + bt_gu - 1) / bt_gu, (count + bt_d - 1) / bt_d};
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
    if (e < E) out[i][e + 1] = before + v[i];
    if (e == 0) out[i][0] = 0;
  }
}

}  // namespace

// Stable rank of each copy among the copies of its expert in this chunk of 1024: lanes of one warp by match, warps by a
// scan of their counts.  The counts of the chunk go to hist; a single chunk writes the tables here as well.
__global__ void __launch_bounds__(kChunk) rank_kernel(const int32_t* ids, int A, int E, Plan t, int single,
                                                      int bt_gu, int bt_d) {
  extern __shared__ uint16_t wcnt[];  // [32][E]
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < 32 * E; i += kChunk) wcnt[i] = 0;
  __syncthreads();
  const long long a = (long long)blockIdx.x * kChunk + threadIdx.x;
  int e = a < A ? ids[a] : -1;
  if (e < 0 || e >= E) e = -1;
  const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e);
  const int below = __popc(peers & ((1u << lane) - 1u));
  if (e >= 0 && below == 0) wcnt[warp * E + e] = (uint16_t)__popc(peers);
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kChunk) {
    int sum = 0;
    for (int w = 0; w < 32; ++w) {
      const int v = wcnt[w * E + i];
      wcnt[w * E + i] = (uint16_t)sum;
      sum += v;
    }
    t.hist[(size_t)blockIdx.x * E + i] = sum;
  }
  __syncthreads();
  if (a < A) t.rank[a] = e < 0 ? -1 : wcnt[warp * E + e] + below;
  if (single) place_tables(t, E, 1, bt_gu, bt_d);
}

__global__ void __launch_bounds__(1024) place_kernel(Plan t, int E, int chunks, int bt_gu, int bt_d) {
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  place_tables(t, E, chunks, bt_gu, bt_d);
}

// Quantizes each token once and writes it to the sorted rows of all its copies (the layout of fp8_quantize_kernel: one
// warp per 512 columns of a token).
template <int DT>
__global__ void __launch_bounds__(256) scatter_kernel(const uint16_t* x, const int32_t* ids,
                                                      int M, int E, int topk, int K, int SW, Plan t,
                                                      uint8_t* codes, uint32_t* scales) {
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
    uint32_t word = 0;
    uint2 c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = w * 512 + h * 256 + lane * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (k < K) v = ldg_stream(x + row * K + k);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
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
      c[h].x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
      c[h].y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
      word |= (b | (__shfl_sync(0xFFFFFFFFu, b, 16) << 8)) << (16 * h);  // lane 0's word: the blocks of lanes 0 and 16
    }
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
}

// y_m = round(sum_j w_mj d[pos_mj]), slots in order, 32 bits until the end.  One thread per 4 columns of a token.
__global__ void __launch_bounds__(256) combine_kernel(const float* d, const int* pos,
                                                      const float* weights, int M, int topk, int N, int dt,
                                                      uint16_t* y) {
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int cols = (N + 3) / 4;
  const long long items = (long long)M * cols;
  const bool wide = (N & 3) == 0;
  for (long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x; it < items;
       it += (long long)gridDim.x * blockDim.x) {
    const long long m = it / cols;
    const int n = (int)(it - m * cols) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < topk; ++j) {
      const int r = pos[m * topk + j];
      if (r < 0) continue;
      const float w = weights[m * topk + j];
      const float* src = d + (size_t)r * N + n;
      float4 v;
      if (wide) v = *reinterpret_cast<const float4*>(src);
      else v = make_float4(src[0], n + 1 < N ? src[1] : 0.f, n + 2 < N ? src[2] : 0.f, n + 3 < N ? src[3] : 0.f);
      s.x = fmaf(w, v.x, s.x);
      s.y = fmaf(w, v.y, s.y);
      s.z = fmaf(w, v.z, s.z);
      s.w = fmaf(w, v.w, s.w);
    }
    uint16_t* o = y + m * N + n;
    const float f[4] = {s.x, s.y, s.z, s.w};
    if (wide) {
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
  if (cnt > 48 * 1024 &&
      cudaFuncSetAttribute(rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess)
    return AWQ_ERR_CUDA;
  cudaError_t e = launch_pdl(rank_kernel, dim3((unsigned)chunks), dim3(kChunk), cnt, a.st, a.ids, A, a.E, t,
                             chunks == 1 ? 1 : 0, bt_gu, bt_d);
  if (e == cudaSuccess && chunks > 1)
    e = launch_pdl(place_kernel, dim3(1), dim3(1024), 0, a.st, t, a.E, chunks, bt_gu, bt_d);
  if (e != cudaSuccess) return AWQ_ERR_CUDA;
  const int SW = fp8_scale_cols(a.K) / 4;
  const long long cap = (long long)num_sms() * 8;
  long long blocks = ((long long)a.M * SW + 7) / 8;
  auto scatter = a.dt == AWQ_DTYPE_F16 ? scatter_kernel<AWQ_DTYPE_F16> : scatter_kernel<AWQ_DTYPE_BF16>;
  e = launch_pdl(scatter, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, a.st, a.x, a.ids, a.M, a.E, a.topk,
                 a.K, SW, t, ws + l.xc, reinterpret_cast<uint32_t*>(ws + l.xs));
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
  st = w8a8_launch(down);
  if (st != AWQ_OK) return st;
  blocks = ((long long)a.M * ((a.N + 3) / 4) + 255) / 256;
  e = launch_pdl(combine_kernel, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, a.st,
                 reinterpret_cast<const float*>(ws + l.d), static_cast<const int*>(t.pos), a.weights, a.M, a.topk, a.N,
                 a.dt, a.y);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
