// route.cu -- moe_route: the experts of each token and their weights, from the router's logits.
//
// Scores p = softmax(l) or 1 / (1 + e^-l); the choice goes by q = p + bias.  With groups, a group counts the sum of its
// two largest q, the topk_groups best groups stay, and the topk largest q among their experts are taken, equal values by
// the lowest index.  The weights are the p of the chosen experts (not q), divided by their sum where asked, times scale.
// Comparisons are made in 64 bits: next to a border 32-bit scores would order experts by their rounding.
#include "fp8.cuh"

namespace awq {

namespace {

constexpr double kMaskedChoice = -1e300;  // an expert whose logit is -inf or NaN comes after every other one
constexpr int kRouteWarps = 4;

template <int DT>
__device__ __forceinline__ float route_logit(const void* l, size_t i) {
  if constexpr (DT == AWQ_DTYPE_F32) return static_cast<const float*>(l)[i];
  else if constexpr (DT == AWQ_DTYPE_F16) return __half2float(static_cast<const __half*>(l)[i]);
  else return __bfloat162float(static_cast<const __nv_bfloat16*>(l)[i]);
}

struct RouteParams {
  const void* logits;
  const float* bias;
  int M, E, topk, score, groups, topk_groups, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

}  // namespace

// One warp per token; lane l holds experts l, l + 32, ... (NE of them).
template <int DT, int NE>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p) {
  extern __shared__ double route_q[];  // [warps][E]: the choices, for the group sums
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double* qs = route_q + (size_t)warp * p.E;
  for (long long m = (long long)blockIdx.x * kRouteWarps + warp; m < p.M; m += (long long)gridDim.x * kRouteWarps) {
    double s[NE], q[NE];
    float l[NE];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 32 + lane;
      float v = -INFINITY;
      if (e < p.E) v = route_logit<DT>(p.logits, (size_t)m * p.E + e);
      v = v != v ? -INFINITY : fminf(v, 3.402823466e38f);
      l[i] = v;
      top = fmaxf(top, v);
    }
    if (p.score == AWQ_SCORE_SOFTMAX) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        s[i] = l[i] == -INFINITY ? 0.0 : exp((double)l[i] - (double)top);
        sum += s[i];
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = l[i] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 32 + lane;
      q[i] = -INFINITY;  // a bias of -inf or NaN masks in the choice as well
      if (e < p.E)
        q[i] = l[i] == -INFINITY ? kMaskedChoice : fmax(s[i] + (p.bias ? (double)p.bias[e] : 0.0), kMaskedChoice);
    }
    if (p.groups > 1) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (i * 32 + lane < p.E) qs[i * 32 + lane] = q[i];
      __syncwarp();
      const int per = p.E / p.groups;
      double v = -INFINITY;
      if (lane < p.groups) {
        double a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < per; ++i) {
          const double x = qs[lane * per + i];
          if (x > a) { b = a; a = x; }
          else if (x > b) b = x;
        }
        v = per > 1 ? a + b : a;
      }
      int before = 0;  // groups that come before this lane's
      for (int g = 0; g < p.groups; ++g) {
        const double o = __shfl_sync(0xFFFFFFFFu, v, g);
        before += (o > v || (o == v && g < lane)) ? 1 : 0;
      }
      const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < p.groups && before < p.topk_groups);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = i * 32 + lane;
        if (e < p.E && !((kept >> (e / per)) & 1u)) q[i] = -INFINITY;
      }
    }
    uint32_t taken = 0;  // bit i: this lane's expert i is taken
    double mine = 0.0, total = 0.0;
    int id = 0;
    for (int k = 0; k < p.topk; ++k) {
      double bq = -INFINITY, bs = 0.0;
      int be = 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = i * 32 + lane;
        if (!((taken >> i) & 1u) && e < p.E && q[i] > bq) {
          bq = q[i];
          bs = s[i];
          be = e;
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const double oq = __shfl_xor_sync(0xFFFFFFFFu, bq, d);
        const double os = __shfl_xor_sync(0xFFFFFFFFu, bs, d);
        const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, d);
        if (oq > bq || (oq == bq && oe < be)) {
          bq = oq;
          bs = os;
          be = oe;
        }
      }
      if ((be & 31) == lane) taken |= 1u << (be >> 5);
      if (lane == k) {
        mine = bs;
        id = be;
      }
      total += bs;
    }
    if (lane < p.topk) {
      const double w = p.renorm ? (total > 0.0 ? mine / total : 0.0) : mine;
      p.ids[(size_t)m * p.topk + lane] = id;
      p.weights[(size_t)m * p.topk + lane] = (float)(w * (double)p.scale);
    }
  }
}

template <int DT>
static cudaError_t route_pick(const RouteParams& p, unsigned grid, size_t smem, cudaStream_t st) {
  const int per_lane = (p.E + 31) / 32;
  auto kernel = per_lane <= 1   ? route_kernel<DT, 1>
                : per_lane <= 2 ? route_kernel<DT, 2>
                : per_lane <= 4 ? route_kernel<DT, 4>
                : per_lane <= 8 ? route_kernel<DT, 8>
                : per_lane <= 16 ? route_kernel<DT, 16>
                                 : route_kernel<DT, 32>;
  return launch_pdl(kernel, dim3(grid), dim3(32 * kRouteWarps), smem, st, p);
}

awq_status moe_route_launch(const void* logits, int dt, const float* bias, int M, int E, int topk, int score, int groups,
                            int topk_groups, int renorm, float scale, int32_t* ids, float* weights, cudaStream_t st) {
  const RouteParams p{logits, bias, M, E, topk, score, groups, topk_groups, renorm, scale, ids, weights};
  long long grid = ((long long)M + kRouteWarps - 1) / kRouteWarps;
  const long long cap = (long long)num_sms() * 16;
  if (grid > cap) grid = cap;
  const size_t smem = groups > 1 ? (size_t)kRouteWarps * E * sizeof(double) : 0;  // at most 32 KB
  const cudaError_t e = dt == AWQ_DTYPE_F32   ? route_pick<AWQ_DTYPE_F32>(p, (unsigned)grid, smem, st)
                        : dt == AWQ_DTYPE_F16 ? route_pick<AWQ_DTYPE_F16>(p, (unsigned)grid, smem, st)
                                              : route_pick<AWQ_DTYPE_BF16>(p, (unsigned)grid, smem, st);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
