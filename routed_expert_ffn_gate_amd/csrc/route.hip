// Routing rule on logits: softmax or sigmoid scores, a bias for balance, groups
// of experts, top-k, renormalised weights.
//
// Definition (include/moelb.h, moelb_route): s = scores of z, c = s + bias;
// the groups with the largest scores stay; idx = the k largest c, w = scale s.
//
// A wave per token, four experts a lane, in 64 bits.
#include <float.h>
#include <math.h>

#include "common.h"

namespace {

constexpr int WAVES = 4;

struct RouteArgs {
  const float* z;
  const float* bias;
  int32_t* idx;
  float* wts;
  float* gap;
  int T, E, k, sigmoid, groups, topk_groups, group_top, renorm;
  float scale;
};

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <class V, class Op>
__device__ __forceinline__ V wave_all(V v, Op op) {
#pragma unroll
  for (int o = 1; o < MOELB_WAVE; o <<= 1) v = op(v, __shfl_xor(v, o, MOELB_WAVE));
  return v;
}

// One token by one wave; cs holds E and gs `groups` doubles of LDS.
__device__ __forceinline__ void route_token(const RouteArgs& p, int t, double* cs, double* gs) {
  const int lane = threadIdx.x & 63;
  auto add = [](double a, double b) { return a + b; };
  auto larger = [](double a, double b) { return a > b ? a : b; };
  double z[4], s[4], c[4], key[4];
  bool on[4];
  double top = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = lane + 64 * q;
    const float v = e < p.E ? p.z[(size_t)t * p.E + e] : -INFINITY;
    on[q] = v > -INFINITY;  // neither -inf nor NaN
    z[q] = on[q] ? (double)fminf(v, FLT_MAX) : -INFINITY;
    top = larger(top, z[q]);
  }
  if (p.sigmoid) {
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = on[q] ? 1.0 / (1.0 + exp(-z[q])) : 0.0;
  } else {
    top = wave_all(top, larger);
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      s[q] = on[q] ? exp(z[q] - top) : 0.0;
      sum += s[q];
    }
    sum = wave_all(sum, add);
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = on[q] ? s[q] / sum : 0.0;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = lane + 64 * q;
    c[q] = on[q] ? s[q] : -INFINITY;
    if (p.bias && on[q]) {
      const double v = s[q] + (double)p.bias[e];
      c[q] = v > -INFINITY ? (v < (double)FLT_MAX ? v : (double)FLT_MAX) : -INFINITY;
    }
    key[q] = p.bias ? c[q] : z[q];
  }
  if (p.groups > 1) {
    const int size = p.E / p.groups;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (lane + 64 * q < p.E) cs[lane + 64 * q] = c[q];
    wave_fence();
    for (int g = lane; g < p.groups; g += MOELB_WAVE) {
      double a = -INFINITY, b = -INFINITY;  // the group's largest and second largest
      for (int i = 0; i < size; ++i) {
        const double v = cs[g * size + i];
        b = v > a ? a : larger(b, v);
        a = larger(a, v);
      }
      gs[g] = p.group_top == 1 ? a : a + b;
    }
    wave_fence();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int g = min((lane + 64 * q) / size, p.groups - 1);
      const double mine = gs[g];
      int before = 0;
      for (int f = 0; f < p.groups; ++f) before += gs[f] > mine || (gs[f] == mine && f < g);
      if (before >= p.topk_groups) c[q] = key[q] = -INFINITY;
    }
    wave_fence();
  }
  // k + 1 maxima; lane j keeps pick j
  int my_id = -1;
  double my_s = 0.0, my_c = -INFINITY;
  for (int j = 0; j <= p.k; ++j) {
    double best = -INFINITY;
    int id = 1 << 20;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (key[q] > best) best = key[q], id = lane + 64 * q;
#pragma unroll
    for (int o = 1; o < MOELB_WAVE; o <<= 1) {
      const double ob = __shfl_xor(best, o, MOELB_WAVE);
      const int oi = __shfl_xor(id, o, MOELB_WAVE);
      if (ob > best || (ob == best && oi < id)) best = ob, id = oi;
    }
    if (best == -INFINITY) break;  // the same in every lane
    double ss = 0.0, cc = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (id == lane + 64 * q) ss = s[q], cc = c[q], key[q] = -INFINITY;
    ss = __shfl(ss, id & 63, MOELB_WAVE);
    cc = __shfl(cc, id & 63, MOELB_WAVE);
    if (lane == j) my_id = id, my_s = ss, my_c = cc;
  }
  double total = wave_all(lane < p.k ? my_s : 0.0, add);
  const double f = p.renorm ? (double)p.scale / (total + 1e-20) : (double)p.scale;
  if (lane < p.k) {
    p.idx[(size_t)t * p.k + lane] = my_id;
    if (p.wts) p.wts[(size_t)t * p.k + lane] = (float)(my_s * f);
  }
  if (p.gap) {
    const double next = __shfl_down(my_c, 1, MOELB_WAVE);
    if (lane == p.k - 1) p.gap[t] = next > -INFINITY ? (float)(my_c - next) : INFINITY;
  }
}

__global__ __launch_bounds__(WAVES * MOELB_WAVE) void route_kernel(RouteArgs p) {
  __shared__ double cs[WAVES][MOELB_MAX_E], gs[WAVES][MOELB_MAX_E];
  const int wave = threadIdx.x >> 6;
  for (long long t = (long long)blockIdx.x * WAVES + wave; t < p.T; t += (long long)gridDim.x * WAVES)
    route_token(p, (int)t, cs[wave], gs[wave]);
}

}  // namespace

extern "C" int moelb_route(const float* z, int T, int E, int k, int score, const float* bias, int groups,
                           int topk_groups, int group_top, int renorm, float scale, int32_t* idx, float* wts,
                           float* gap, void* stream) {
  if (T < 0 || E < 1 || E > MOELB_MAX_E || k < 1 || k > MOELB_MAX_K || k > E) return MOELB_EINVAL;
  if (score != MOELB_SCORE_SOFTMAX && score != MOELB_SCORE_SIGMOID) return MOELB_EINVAL;
  if (groups < 1 || groups > E || E % groups != 0 || topk_groups < 1 || topk_groups > groups) return MOELB_EINVAL;
  if (topk_groups * (E / groups) < k || group_top < 1 || group_top > 2 || group_top > E / groups) return MOELB_EINVAL;
  if (!(fabsf(scale) <= FLT_MAX)) return MOELB_EINVAL;
  if (T == 0) return MOELB_OK;
  if (!z || !idx) return MOELB_EINVAL;
  RouteArgs p = {z, bias, idx, wts, gap, T, E, k, score == MOELB_SCORE_SIGMOID, groups, topk_groups, group_top,
                 renorm != 0, scale};
  const size_t blocks = ((size_t)T + WAVES - 1) / WAVES, most = moelb_most_blocks(WAVES * MOELB_WAVE);
  hipLaunchKernelGGL(route_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(WAVES * MOELB_WAVE), 0,
                     static_cast<hipStream_t>(stream), p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}
