// route.cu -- moe_route: the experts of each token and their weights, from the router's logits.
//
// Scores p = softmax(l) or 1 / (1 + e^-l); the choice goes by q = p + bias.  With groups, a group counts the sum of its
// two largest q, the topk_groups best groups stay, and the topk largest q among their experts are taken, equal values by
// the lowest index.  The weights are the p of the chosen experts (not q), divided by their sum where asked, times scale.
// The order is that of the 64-bit values: next to a border 32-bit scores would order experts by their rounding.  A warp
// works in 32 bits and looks at the gaps that its choice rests on.  Where each is wider than the scores' error (or the two
// experts have the same logit and bias, a true tie), the 64-bit order is the same; where one is not, the few experts in
// question are compared in 64 bits; where a border between groups is in doubt, the group sums are, or the warp does the token again
// in 64 bits.  Between the chosen the errors of two neighbours count.  What is left out is held against the largest error in the
// row: with a bias an expert far behind may have a large score, and a group two large choices that cancel.
// The weights are 32-bit values of the chosen experts' scores.
// Bound by latency for few tokens (one token among 256 experts: 4.8 us) and by issue slots for many (8192 tokens: 19 us, 1615
// instructions per token at 63 % of the issue rate; its 8.9 MB would take 1.4).  All in 64 bits it took 34 us; a
// token done again in 64 bits for one doubtful gap cost 8 us of tail per call, which the comparisons in place avoid.
#include "fp8.cuh"

namespace awq {

namespace {

constexpr double kMaskedChoice = -1e300;  // an expert whose logit is -inf or NaN comes after every other one
constexpr int kRouteWarps = 4;
constexpr float kMasked32 = -3.402823466e38f;
constexpr float kLeastBias = -1e30f;  // a smaller bias (or NaN) masks its expert in the choice as well

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
  int share;  // lanes per group: the largest power of two with share * groups <= 32
  float scale;
  int32_t* ids;
  float* weights;
};

}  // namespace

__device__ __forceinline__ float route_clean(float v) {  // a logit as it counts: NaN is -inf, +inf the largest number
  return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}
// The score in 64 bits (softmax: the row's largest logit and 64-bit sum).
__device__ __forceinline__ double route_score(const RouteParams& p, float l, float top, double sum) {
  if (l == -INFINITY) return 0.0;
  if (p.score == AWQ_SCORE_SOFTMAX) return exp((double)l - (double)top) / sum;
  return 1.0 / (1.0 + exp(-(double)l));
}

// One token in 64 bits, the choices in shared memory (qs [E], the warp's own): few registers, so that this rare path
// does not cost the usual one its occupancy.
template <int DT>
__device__ __noinline__ void route_exact(const RouteParams& p, long long m, double* qs) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
#pragma unroll 4
  for (int e = lane; e < p.E; e += 32) top = fmaxf(top, route_clean(route_logit<DT>(p.logits, (size_t)m * p.E + e)));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  double sum = 0.0;
  if (p.score == AWQ_SCORE_SOFTMAX) {
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32)
      sum += route_score(p, route_clean(route_logit<DT>(p.logits, (size_t)m * p.E + e)), top, 1.0);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  }
#pragma unroll 4
  for (int e = lane; e < p.E; e += 32) {
    const float l = route_clean(route_logit<DT>(p.logits, (size_t)m * p.E + e));
    const float b = p.bias ? p.bias[e] : 0.f;
    qs[e] = l == -INFINITY || !(b >= kLeastBias) ? kMaskedChoice : route_score(p, l, top, sum) + (double)b;
  }
  __syncwarp();
  if (p.groups > 1) {
    const int per = p.E / p.groups;
    double v = -INFINITY;
    if (lane < p.groups) {
      double a = -INFINITY, b = -INFINITY;
#pragma unroll 8
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
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32)
      if (!((kept >> (e / per)) & 1u)) qs[e] = -INFINITY;
    __syncwarp();
  }
  int id = 0;
  for (int k = 0; k < p.topk; ++k) {
    double bq = -INFINITY;
    int be = 0x7FFFFFFF;
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32)
      if (qs[e] > bq) {
        bq = qs[e];
        be = e;
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double oq = __shfl_xor_sync(0xFFFFFFFFu, bq, d);
      const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, d);
      if (oq > bq || (oq == bq && oe < be)) {
        bq = oq;
        be = oe;
      }
    }
    if ((be & 31) == lane) qs[be] = -INFINITY;
    if (lane == k) id = be;
    __syncwarp();
  }
  double w = 0.0;
  if (lane < p.topk) w = route_score(p, route_clean(route_logit<DT>(p.logits, (size_t)m * p.E + id)), top, sum);
  if (p.renorm) {
    double total = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (lane < p.topk) {
    p.ids[(size_t)m * p.topk + lane] = id;
    p.weights[(size_t)m * p.topk + lane] = (float)(w * (double)p.scale);
  }
  __syncwarp();
}

// fp32 as an unsigned whole number in the same order.
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float route_unkey(uint32_t k) {
  return __uint_as_float(k ^ (~(uint32_t)((int)k >> 31) | 0x80000000u));
}

// The two largest of a group, from the two largest of its halves.
__device__ __forceinline__ void route_top2(float& a, float& b, float oa, float ob) {
  b = fmaxf(fminf(a, oa), fmaxf(b, ob));
  a = fmaxf(a, oa);
}

// One warp per token; lane l holds experts l, l + 32, ... (NE of them).
template <int DT, int NE>
__global__ void __launch_bounds__(32 * kRouteWarps, NE <= 4 ? 8 : NE <= 8 ? 5 : NE <= 16 ? 4 : 2) route_kernel(const RouteParams p) {
  extern __shared__ double route_q[];  // [warps][E + 32]: the choices, for the group sums and the 64-bit path
  pdl_launch_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool softmax = p.score == AWQ_SCORE_SOFTMAX;
  double* own = route_q + (size_t)warp * (p.E + 32);
  float* qs = reinterpret_cast<float*>(own);
  float bias[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) bias[i] = 0.f;
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < NE; ++i) bias[i] = p.bias[min(i * 32 + lane, p.E - 1)];
  }
  const int per = p.E / p.groups, share = p.share;  // experts and lanes per group
  const float per_inv = 1.f / (float)per;
  for (long long m = (long long)blockIdx.x * kRouteWarps + warp; m < p.M; m += (long long)gridDim.x * kRouteWarps) {
    float l[NE], q[NE];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      l[i] = route_logit<DT>(p.logits, (size_t)m * p.E + min(i * 32 + lane, p.E - 1));  // all loads at once
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      l[i] = i * 32 + lane >= p.E || l[i] != l[i] ? -INFINITY : fminf(l[i], 3.402823466e38f);
      top = fmaxf(top, l[i]);
    }
    float total = 1.f;
    if (softmax) {
      top = route_unkey(__reduce_max_sync(0xFFFFFFFFu, route_key(top)));
      total = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        q[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - top);
        total += q[i];
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    }
    const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float s = softmax ? q[i] * inv : __fdividef(1.f, 1.f + expf(-l[i]));
      q[i] = l[i] == -INFINITY || !(bias[i] >= kLeastBias) ? kMasked32 : s + bias[i];
      if (i * 32 + lane >= p.E) q[i] = -INFINITY;
    }
    bool doubt = false;
    if (p.groups > 1) {
      // Group g's choices stand at g * pitch: the pitch moves each group by its lanes' banks, so that no two lanes meet.
      const int pitch = per + share;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = i * 32 + lane;
        const int of = (int)(((float)e + 0.5f) * per_inv);  // e / per: below 1024 the half keeps the product off whole numbers
        if (e < p.E) qs[e + of * share] = q[i];
      }
      __syncwarp();
      const int g = lane >> (__ffs(share) - 1);
      const bool group = g < p.groups;
      float a = -INFINITY, b = -INFINITY;
      if (group) {
        const float* end = qs + g * pitch + per;
#pragma unroll 8
        for (const float* x = qs + g * pitch + (lane & (share - 1)); x < end; x += share) route_top2(a, b, *x, -INFINITY);
      }
      for (int d = 1; d < share; d <<= 1)
        route_top2(a, b, __shfl_xor_sync(0xFFFFFFFFu, a, d), __shfl_xor_sync(0xFFFFFFFFu, b, d));
      const float v = per > 1 ? a + b : a;
      // Bounds every group's sum and the two scores in it (0 .. 1).  The largest counts for all: a group whose large choices
      // cancel may stand anywhere in the order with its error.
      float size = group ? fabsf(a) + (per > 1 ? fabsf(b) : 0.f) + 2.f : 0.f;
      size = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(size)));
      int before = 0;  // groups that come before this lane's
      bool near = false;
      for (int o = 0; o < p.groups; ++o) {
        const float w = __shfl_sync(0xFFFFFFFFu, v, o * share);
        before += (w > v || (w == v && o < g)) ? 1 : 0;
        near |= o != g && !(fabsf(w - v) > (softmax ? 0x1p-17f : 0x1p-20f) * size);
      }
      // The border is in doubt where the last group in or the first one out has a neighbour within the error: where the two are
      // further apart than that, no group changes sides.
      doubt = group && near && p.topk_groups < p.groups && (before == p.topk_groups - 1 || before == p.topk_groups);
      if (__any_sync(0xFFFFFFFFu, doubt) && !softmax) {
        // The groups' sums in 64 bits, where each group's two largest are clear of its third (or the whole token again).
        float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY;
        int i0 = 0, i1 = 0;
        if (group) {
#pragma unroll 8
          for (int i = 0; i < per; ++i) {
            const float x = qs[g * pitch + i];
            t2 = fmaxf(t2, fminf(x, t1));
            if (x > t0) {
              t1 = t0;
              i1 = i0;
              t0 = x;
              i0 = i;
            } else if (x > t1) {
              t1 = x;
              i1 = i;
            }
          }
        }
        double sum = -INFINITY;
        doubt = false;
        if (group) {
          auto choice = [&](int i) {
            const int e = g * per + i;
            const float l0 = route_clean(route_logit<DT>(p.logits, (size_t)m * p.E + e)), b0 = p.bias ? p.bias[e] : 0.f;
            return l0 == -INFINITY || !(b0 >= kLeastBias) ? kMaskedChoice : route_score(p, l0, 0.f, 1.0) + (double)b0;
          };
          sum = choice(i0);
          if (per > 1) sum += choice(i1);
          doubt = per > 2 && !(t1 - t2 > 0x1p-20f * 2.f + 0x1p-22f * (fabsf(t1) + fabsf(t2)));
        }
        before = 0;
        for (int o = 0; o < p.groups; ++o) {
          const double w = __shfl_sync(0xFFFFFFFFu, sum, o * share);
          before += (w > sum || (w == sum && o < g)) ? 1 : 0;
        }
      }
      const uint32_t kept = __ballot_sync(0xFFFFFFFFu, group && before < p.topk_groups);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = i * 32 + lane;
        const int of = (int)(((float)e + 0.5f) * per_inv);
        if (e < p.E && !((kept >> (of * share)) & 1u)) q[i] = -INFINITY;
      }
    }
    float mine = -INFINITY;  // lane k: the k-th largest choice; lane topk: the first one left out
    int id = 0, count = 0;
    // Each lane knows its two largest (the first places among equals); the lane that gives one moves up, and when one has
    // given both, all look again.
    float b0, b1;
    int i0, i1, known;
    uint32_t gone = 0;  // bit i: this lane's expert i is taken
    auto look = [&]() {
      b0 = b1 = -INFINITY;
      i0 = i1 = 0;
      known = 2;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float x = (gone >> i) & 1u ? -INFINITY : q[i];
        if (x > b0) {
          b1 = b0;
          i1 = i0;
          b0 = x;
          i0 = i;
        } else if (x > b1) {
          b1 = x;
          i1 = i;
        }
      }
    };
    look();
    auto take = [&]() {  // the next one, the lowest index among equals; false if none is left or no lane
      const float bq = route_unkey(__reduce_max_sync(0xFFFFFFFFu, route_key(b0)));
      if (count == 32 || bq == -INFINITY) return false;
      const uint32_t own_at = (uint32_t)(i0 * 32 + lane);
      const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, b0 == bq ? own_at : 0xFFFFFFFFu);
      if (lane == count) {
        mine = bq;
        id = (int)e;
      }
      if (e == own_at) {
        gone |= 1u << i0;
        b0 = b1;
        i0 = i1;
        b1 = -INFINITY;
        --known;
      }
      if (__any_sync(0xFFFFFFFFu, known == 0)) look();
      ++count;
      return true;
    };
    bool more = true;  // something may be left that has not been taken
    while (count <= p.topk && (more = take())) {}
    // Each choice against the next: a gap within the error of both, between experts of different logit or bias, is in doubt.
    float lk, bk;
    auto inputs = [&]() {
      lk = lane < count ? route_logit<DT>(p.logits, (size_t)m * p.E + id) : 0.f;
      bk = lane < count && p.bias ? p.bias[id] : 0.f;
      if (lk != lk) lk = -INFINITY;
    };
    inputs();
    const float ln = __shfl_down_sync(0xFFFFFFFFu, lk, 1), bn = __shfl_down_sync(0xFFFFFFFFu, bk, 1);
    const float qn = __shfl_down_sync(0xFFFFFFFFu, mine, 1);
    // A sigmoid's error is below 2^-21 of it (the exponential 2^-22, the sum 2^-24, the quotient 2^-22).  A softmax's is
    // below 2^-16: l - top rounds to 2^-24 of itself, which the exponential takes over (|l - top| < 104 where it is not 0),
    // and the sum of up to 1024 terms to 37 * 2^-24.  A biased score rounds to 2^-24 of itself once more.
    const float rel = softmax ? 0x1p-16f : 0x1p-20f;
    const float most = softmax ? inv : 1.f;  // no score of the row is larger
    bool order = false;  // the order of this one and the next is in doubt
    if (lane < count - 1 && lane < p.topk && mine != kMasked32) {
      // At the border a true tie is in doubt as well: an expert of another logit may stand behind it at the same 32-bit value.
      const bool edge = lane == p.topk - 1, tie = lk == ln && bk == bn && !edge;
      // Among the chosen two neighbours' errors are enough, since the doubt of any of them has all compared.  The last one in
      // stands against all that are out: without a bias their scores, and so their errors, are smaller still; with one, a
      // larger score that its bias lowers may stand anywhere behind, with an error of the largest score's.
      const float of = edge && p.bias ? 2.f * most : fabsf(mine - bk) + fabsf(qn - bn);
      order = !tie && !(mine - qn > rel * of + 0x1p-22f * (fabsf(mine) + fabsf(qn)));
    }
    const uint32_t unsure = __ballot_sync(0xFFFFFFFFu, order);
    bool again = __any_sync(0xFFFFFFFFu, doubt);
    if (unsure >> (p.topk - 1) & 1u) {
      // The border itself: take on until the last one taken is clearly below it, and with it whatever stands behind.
      const float edge = __shfl_sync(0xFFFFFFFFu, mine, p.topk - 1);
      for (;;) {
        const float last = __shfl_sync(0xFFFFFFFFu, mine, count - 1);
        if (edge - last > rel * 2.f * most + 0x1p-22f * (fabsf(edge) + fabsf(last))) break;
        if (!(more = take())) {
          again |= count == 32;
          break;
        }
      }
      inputs();
    }
    if (p.topk == 32) {  // no lane for the first one left out
      const float best = route_unkey(__reduce_max_sync(0xFFFFFFFFu, route_key(b0)));
      const float edge = __shfl_sync(0xFFFFFFFFu, mine, 31);
      again |= best != -INFINITY && edge != kMasked32 && !(edge - best > rel * 2.f * most + 0x1p-22f * (fabsf(edge) + fabsf(best)));
    }
    if (again) {
      __syncwarp();
      route_exact<DT>(p, m, own);
      continue;
    }
    const bool has = lane < p.topk;
    lk = route_clean(lk);
    if (unsure == 0) {  // the order stands: 32 bits do for the weights, unless nearly nothing is to be divided by itself
      float w = 0.f;
      if (has && lk != -INFINITY) w = softmax ? expf(lk - top) : 1.f / (1.f + expf(-lk));
      float of = softmax ? total : 1.f;
      if (p.renorm) {
        of = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) of += __shfl_xor_sync(0xFFFFFFFFu, of, d);
      }
      if (!p.renorm || of > 0x1p-20f) {
        if (has) {
          p.ids[(size_t)m * p.topk + lane] = id;
          p.weights[(size_t)m * p.topk + lane] = (of > 0.f ? w / of : 0.f) * p.scale;
        }
        continue;
      }
    }
    // The scores of the taken in 64 bits.
    double sum = 1.0, w = 0.0;
    if (softmax && (!p.renorm || unsure)) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) sum += l[i] == -INFINITY ? 0.0 : exp((double)l[i] - (double)top);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    }
    if (lane < count) w = route_score(p, lk, top, sum);
    if (unsure) {  // in their true order
      const double x = lane >= count ? -INFINITY : mine == kMasked32 ? kMaskedChoice : w + (double)bk;
      int before = 0;
      for (int j = 0; j < count; ++j) {
        const double o = __shfl_sync(0xFFFFFFFFu, x, j);
        const int oi = __shfl_sync(0xFFFFFFFFu, id, j);
        before += (o > x || (o == x && oi < id)) ? 1 : 0;
      }
      int from = lane;
      for (int j = 0; j < p.topk; ++j) {
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, lane < count && before == j);
        if (lane == j) from = __ffs((int)who) - 1;
      }
      id = __shfl_sync(0xFFFFFFFFu, id, from);
      w = __shfl_sync(0xFFFFFFFFu, w, from);
    }
    if (!has) w = 0.0;
    if (p.renorm) {
      double total64 = w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total64 += __shfl_xor_sync(0xFFFFFFFFu, total64, d);
      w = total64 > 0.0 ? w / total64 : 0.0;
    }
    if (has) {
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
  int share = 32;
  while (share * groups > 32) share /= 2;
  const RouteParams p{logits, bias, M, E, topk, score, groups, topk_groups, renorm, share, scale, ids, weights};
  long long grid = ((long long)M + kRouteWarps - 1) / kRouteWarps;
  const long long cap = (long long)num_sms() * 16;
  if (grid > cap) grid = cap;
  const size_t smem = (size_t)kRouteWarps * (E + 32) * sizeof(double);  // at most 33 KB
  const cudaError_t e = dt == AWQ_DTYPE_F32   ? route_pick<AWQ_DTYPE_F32>(p, (unsigned)grid, smem, st)
                        : dt == AWQ_DTYPE_F16 ? route_pick<AWQ_DTYPE_F16>(p, (unsigned)grid, smem, st)
                                              : route_pick<AWQ_DTYPE_BF16>(p, (unsigned)grid, smem, st);
  return e == cudaSuccess ? AWQ_OK : AWQ_ERR_CUDA;
}

}  // namespace awq
