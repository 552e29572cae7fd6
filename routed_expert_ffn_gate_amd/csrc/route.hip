// Routing rule on logits: softmax or sigmoid scores, a bias for balance, groups
// of experts, top-k, renormalised weights.
//
// Definition (include/moelb.h, moelb_route): s = scores of z, c = s + bias;
// the groups with the largest scores stay; idx = the k largest c, w = scale s.
//
// Forms of the same rule:
//  * route_fast: eight lanes a token, in fp32.  Values become 24-bit fixed-point
//    keys with the id below (larger value, then lower id), and the k + 2 largest
//    are kept by an insertion list, one v_med3_u32 an entry; the lanes' lists are
//    merged by DPP.  It also finds where fp32 cannot tell.
//  * Two of the first k + 1 keys nearer than their error bounds: the listed experts
//    are ranked in 64 bits by the token's eight lanes.
//  * Groups nearer to the border of the kept ones than the errors of their own best
//    two: a sigmoid's by those two in 64 bits.
//  * What that does not decide (ties beyond the list or the two, a softmax's groups,
//    values below the keys' window): route_token, a whole wave a token, four
//    experts a lane, in 64 bits.
// So the picks are those of 64-bit arithmetic.  Bound by vector instructions (60-70 %
// active): T = 32768, 256 experts, sigmoid, bias, 4 of 8 groups, top 8 in 21 us (7 for
// the logits' bytes); 160 experts, softmax, 3 of 8 groups, top 6 20, of peaked logits
// 13; 128 experts, softmax 11; 512 tokens 4.4.
#include <float.h>
#include <math.h>

#include "topk_list.h"

namespace {

constexpr int WAVES = 4, LPT = 8, TPW = MOELB_WAVE / LPT;  // lanes a token, tokens a wave

struct RouteArgs {
  const float* z;
  const float* bias;
  int32_t* idx;
  float* wts;
  float* gap;
  int T, E, k, sigmoid, groups, topk_groups, group_top, renorm;
  float scale;
  int stride;  // floats of a token's row in LDS (groups > 1)
  int vec;     // rows of z, and bias, can be read 16 bytes at a time
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

// A logit as the rule takes it: masked (-inf, NaN) to -inf, +inf to the largest float.
__device__ __forceinline__ float taken(float v) { return fminf(fmaxf(v, -INFINITY), FLT_MAX); }

// The median; with a NaN among them the least of the others.  (The builtin with
// constant operands is folded to forms that treat a NaN otherwise.)
__device__ __forceinline__ float med3(float a, float b, float c) {
  float r;
  asm("v_med3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// ---------------------------------------------------------------- 64 bits

// The wave's largest, in every lane: rotations within 16 lanes, then the halves'
// and quarters' exchange (no LDS round trip).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto ror = [&](auto n) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + decltype(n)::value, 0xf, 0xf, true);
    v = o > v ? o : v;
  };
  ror(std::integral_constant<int, 8>{});
  ror(std::integral_constant<int, 4>{});
  ror(std::integral_constant<int, 2>{});
  ror(std::integral_constant<int, 1>{});
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = a[0] > a[1] ? a[0] : a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return b[0] > b[1] ? b[0] : b[1];
}

// A double's bits as an unsigned integer in the doubles' order (no NaN, -0 as 0);
// -inf is below every other and not 0.
__device__ __forceinline__ uint64_t ordered64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}

// One token by one wave; cs holds E and gs `groups` doubles of LDS (groups > 1).
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
    z[q] = (double)taken(e < p.E ? p.z[(size_t)t * p.E + e] : -INFINITY);
    on[q] = z[q] > -INFINITY;
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
      for (int i = 0; i < size; i += 4) {
        double v[4];  // four reads ahead of their use
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = cs[g * size + min(i + q, size - 1)];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (i + q < size) {
            b = v[q] > a ? a : larger(b, v[q]);
            a = larger(a, v[q]);
          }
      }
      gs[g] = p.group_top == 1 ? a : a + b;
    }
    wave_fence();
    double mine[4];
    int g[4], before[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      g[q] = min((lane + 64 * q) / size, p.groups - 1);
      mine[q] = gs[g[q]];
    }
    for (int f = 0; f < p.groups; f += 4) {
      double o[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) o[n] = gs[min(f + n, p.groups - 1)];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          before[q] += f + n < p.groups && (o[n] > mine[q] || (o[n] == mine[q] && f + n < g[q]));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (before[q] >= p.topk_groups) c[q] = key[q] = -INFINITY;
    wave_fence();
  }
  // k + 1 maxima; lane j keeps pick j
  int my_id = -1;
  double my_s = 0.0, my_c = -INFINITY;
  uint64_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) u[q] = key[q] > -INFINITY ? ordered64(key[q]) : 0ull;
  for (int j = 0; j <= p.k; ++j) {
    uint64_t best = u[0];
#pragma unroll
    for (int q = 1; q < 4; ++q) best = u[q] > best ? u[q] : best;
    const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
    const uint32_t lo = wave_max_u32((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    best = (uint64_t)hi << 32 | lo;
    if (best == 0ull) break;  // nothing is left, the same in every lane
    int id = -1;
#pragma unroll
    for (int q = 3; q >= 0; --q) {
      const uint64_t b = __ballot(u[q] == best);
      id = b ? __ffsll(static_cast<long long>(b)) - 1 + 64 * q : id;  // the lowest id
    }
    double ss = 0.0, cc = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (id >> 6 == q) ss = s[q], cc = c[q];
      if (id == lane + 64 * q) u[q] = 0ull;
    }
    ss = __shfl(ss, id & 63, MOELB_WAVE);
    cc = __shfl(cc, id & 63, MOELB_WAVE);
    if (lane == j) my_id = id, my_s = ss, my_c = cc;
  }
  const double total = wave_all(lane < p.k ? my_s : 0.0, add);
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

// ---------------------------------------------------------------- fp32

// Over a token's eight lanes; every lane gets the result.
template <class Op>
__device__ __forceinline__ float token_all(float v, Op op) {
  auto step = [&](auto m) {
    v = op(v, __uint_as_float(merge_partner<decltype(m)::value>(__float_as_uint(v))));
  };
  step(std::integral_constant<int, 1>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 4>{});
  return v;
}

// Values to keys: window [top - W, top] to 1 .. 2^24 - 5 in the upper 24 bits,
// what lies below it, and NaN (masked), to 0 there, and 255 - id below.
struct Keys {
  float mul, add;
  __device__ __forceinline__ Keys(float top, float W) : mul(16777210.f / W), add(1.f - (top - W) * mul) {}
  __device__ __forceinline__ uint32_t of(float v, int id) const {
    return ((uint32_t)med3(fmaf(v, mul, add), 0.f, 16777215.f) << 8) | (uint32_t)(255 - id);
  }
};

// -inf to NaN, which maxima, minima and medians pass over.
__device__ __forceinline__ float masked(float v) { return fmaf(v, 0.f, v); }

// Eight tokens by one wave.  `lds`: TPW rows of p.stride floats, then TPW x groups
// scores with their errors and TPW x groups kept groups (groups > 1).  Returns the mask of lanes
// whose token has to be routed in 64 bits (outputs not written).
template <int NV, int KL>
__device__ __forceinline__ uint64_t route_fast(const RouteArgs& p, int t0, float* lds) {
  const int lane = threadIdx.x & 63, sub = lane & (LPT - 1), tok = lane / LPT;
  const size_t t = (size_t)t0 + tok;
  const bool active = t < (size_t)p.T;
  const float* zr = p.z + t * p.E;
  auto larger = [](float a, float b) { return fmaxf(a, b); };
  auto add = [](float a, float b) { return a + b; };
  // expert of this lane's value i: four neighbours at a time, the token's lanes side by side
  auto id_of = [&](int i) { return (i >> 2) * (4 * LPT) + sub * 4 + (i & 3); };
  float v[NV];
#pragma unroll
  for (int j = 0; j < NV / 4; ++j) {
    const int e = id_of(4 * j);
    if (p.vec) {
      float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (active && e < p.E) x = *reinterpret_cast<const float4*>(zr + e);
      v[4 * j] = x.x, v[4 * j + 1] = x.y, v[4 * j + 2] = x.z, v[4 * j + 3] = x.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[4 * j + c] = active && e + c < p.E ? zr[e + c] : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = taken(v[i]);
  float m = 0.f, inv = 0.f;  // softmax: the largest logit and 1 / sum
  if (!p.sigmoid) {
    m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, v[i]);
    m = token_all(m, larger);
    // in a tree, so that its error stays small (see the bounds below)
    float part[NV / 2];
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) part[i] = __expf(v[i] - m) + __expf(v[i + NV / 2] - m);
#pragma unroll
    for (int n = NV / 4; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) part[i] += part[i + n];
    const float sum = token_all(part[0], add);
    inv = sum > 0.f ? 1.0f / sum : 0.f;  // 0: every logit is masked
  }
  auto score = [&](float x) { return p.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-x)) : __expf(x - m) * inv; };
  // what the picks go by: c with a bias, else the logit (the same order, exact);
  // NaN where masked
#pragma unroll
  for (int j = 0; j < NV / 4; ++j) {
    const int e = id_of(4 * j);
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias) {
      if (p.vec) {
        if (e < p.E) {
          const float4 x = *reinterpret_cast<const float4*>(p.bias + e);
          b[0] = x.x, b[1] = x.y, b[2] = x.z, b[3] = x.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = e + c < p.E ? p.bias[e + c] : 0.f;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float x = v[4 * j + c];
        v[4 * j + c] = score(x) + fmaf(x, 0.f, masked(taken(b[c])));
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[4 * j + c] = masked(v[4 * j + c]);
    }
  }
  float top = v[0], low = v[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) top = fmaxf(top, v[i]), low = fminf(low, v[i]);
  top = token_all(top, larger);
  low = token_all(low, [](float a, float b) { return fminf(a, b); });
  const float M = fmaxf(1.f, fabsf(top));
  // c: a window of 2 M, so a key's unit is 2^-23 M; logits: 64
  const float W = p.bias ? 2.f * M : 64.f;
  const Keys keys(top, W);
  // Errors: s of a sigmoid under 2^-22 (0.19 of it from the exponential, 0.75 from
  // the sum and the reciprocal), of a softmax under 14 x 2^-24 (8 additions, the
  // exponentials, the quotient); c has the sum's rounding beside it, under 1.5 x 2^-23
  // M in the window, where |c| <= 3 M.  In units that is 3.5 or 8.5 a key.  Two keys
  // are in order if they are further apart than both, 7 or 17 units, and 2 of their
  // own (half a unit each from the product and sum, under one from dropping the
  // fraction).  Logits are exact: unequal keys are in order.
  const uint32_t near = p.bias ? (p.sigmoid ? 9u : 19u) : 0u;
  // one c with a bias, and room for one more rounding of it and of a sum with it
  auto c_error = [&](float c) { return (p.sigmoid ? 0x1p-22f : 14 * 0x1p-24f) + fabsf(c) * 0x1p-22f; };
  // one s without a bias, of logit x: relative to it, since scores may be of any size.
  // In 2^-24: 2.5 |y| of the exponential's argument y (its rounding, the product with
  // log2 e and that constant's), of a softmax's sum 2.5 times the scores' entropy, at
  // most 5.6, and 8 additions, and a few units of the exponential and the quotient.
  // A sigmoid of x > 0 has no more than one of 0.  2^-120: results under the normals
  auto s_error = [&](float x, float s) {
    const float y = fminf(p.sigmoid ? fmaxf(-x, 0.f) : m - x, 128.f);
    return s > -INFINITY ? fmaf(s * 0x1p-23f, fmaf(1.5f, y, 20.f), 0x1p-120f) : 0.f;
  };
  // a window too far from 0 for its sums (the bound is 2^-24 |top| of error, far
  // under a tenth of the window)
  bool redo = fabsf(top) >= (p.bias ? 1e30f : 1e7f);
  uint32_t l[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) l[i] = 0u;
  if (p.groups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) list_insert<KL>(l, keys.of(v[i], id_of(i)));
  } else {
    float* row = lds + tok * p.stride;
    // a group's score, and how far it can be from its value in 64 bits
    float2* gs = reinterpret_cast<float2*>(lds + TPW * p.stride) + tok * p.groups;
    int* kept = reinterpret_cast<int*>(lds + TPW * (p.stride + 2 * p.groups)) + tok * p.groups;
#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      const int e = id_of(4 * j);
      if (e < p.stride)  // a row ends in whole pieces of four
        *reinterpret_cast<float4*>(row + e) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    wave_fence();
    const int size = p.E / p.groups;
    const bool quads = size % 4 == 0;
    // take(x, i) for the values of group g.  Four reads ahead of their use; each lane
    // starts elsewhere: groups of a power of two would meet on one bank
    auto scan = [&](int g, auto take) {
      auto run = [&](int cnt, auto read, auto use) {
        int i = sub % cnt;
        for (int n = 0; n < cnt; n += 4) {
          decltype(read(0)) x[4];
          int at[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[q] = read(i);
            at[q] = i;
            i = i + 1 < cnt ? i + 1 : 0;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < cnt) use(x[q], at[q]);
        }
      };
      const float* r = row + g * size;
      if (quads)
        run(
            size / 4, [&](int i) { return *reinterpret_cast<const float4*>(r + 4 * i); },
            [&](float4 x, int i) { take(x.x, 4 * i), take(x.y, 4 * i + 1), take(x.z, 4 * i + 2), take(x.w, 4 * i + 3); });
      else
        run(size, [&](int i) { return r[i]; }, take);
    };
    for (int g = sub; g < p.groups; g += LPT) {
      float a = -INFINITY, b = -INFINITY;
      scan(g, [&](float x, int) {
        b = med3(a, b, x);
        a = fmaxf(a, x);
      });
      // c: the bounds above, the bias's rounding by the c itself (a group's best two
      // may lie far below the token's); the sum, and the two ends of the comparison,
      // round by as much again.  Halves: two c of the lowest float stay above -inf
      float ea = 0.f, eb = 0.f;
      if (p.bias) {
        ea = c_error(a), eb = c_error(b);
      } else {
        const float za = a, zb = b;
        a = a > -INFINITY ? score(a) : -INFINITY;
        b = b > -INFINITY ? score(b) : -INFINITY;
        ea = s_error(za, a), eb = s_error(zb, b);
      }
      gs[g] = p.group_top == 1 ? make_float2(0.5f * a, 0.5f * ea) : make_float2(0.5f * a + 0.5f * b, 0.5f * ea + 0.5f * eb);
    }
    wave_fence();
    // a group's place among the others; beyond doubt if it is the same with the
    // errors of both taken off and added
    bool doubt = false;
    for (int g = sub; g < p.groups; g += LPT) {
      const float2 me = gs[g];
      const float x = me.x, lo = x - me.y, hi = x + me.y;
      int before = 0, least = 0, most = 0;
      for (int f = 0; f < p.groups; f += 8) {
        float2 y[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = gs[min(f + q, p.groups - 1)];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const bool in = f + q < p.groups;
          before += in && (y[q].x > x || (y[q].x == x && f + q < g));
          least += in && y[q].x - y[q].y > hi;
          most += in && y[q].x + y[q].y >= lo;  // itself among them
        }
      }
      if (least < p.topk_groups && most > p.topk_groups && x > -INFINITY) doubt = true;
      if (before < p.topk_groups) kept[before] = g;
    }
    wave_fence();
    // Doubtful groups of a sigmoid, one a lane: the sum of their best two in 64 bits,
    // unless a third value is near them.  Left to route_token instead: 22.8 us
    // against 21.0 at T = 32768, 4 of 8 groups of 32 (16.8 without any such token).
    const uint64_t doubts = __ballot(doubt && active);
    if (p.sigmoid && p.groups <= LPT && doubts != 0ull) {
      doubt = false;
      if ((doubts >> (tok * LPT)) & 0xff) {
        double c = -INFINITY;
        if (sub < p.groups && gs[sub].x > -INFINITY) {
          float a = -INFINITY, b = -INFINITY;
          int ia = -1, ib = -1, count = 0;
          scan(sub, [&](float x, int i) {
            if (x > a)
              b = a, ib = ia, a = x, ia = i;
            else if (x > b)
              b = x, ib = i;
          });
          const float last = p.group_top == 1 ? a : b, least = last - 2.f * c_error(last);
          scan(sub, [&](float x, int) { count += x >= least; });
          doubt = p.bias && count > 2;
          auto exact = [&](int i) {
            if (i < 0) return (double)-INFINITY;
            const int e = sub * size + i;
            return 1.0 / (1.0 + exp(-(double)taken(zr[e]))) + (p.bias ? (double)p.bias[e] : 0.0);
          };
          const double ca = exact(ia), cb = exact(ib);
          c = p.group_top == 1 ? (ca > cb ? ca : cb) : ca + cb;
        }
        int before = 0;
        for (int f = 0; f < p.groups; ++f) {
          const double o = __shfl(c, tok * LPT + f, MOELB_WAVE);
          before += o > c || (o == c && f < sub);
        }
        if (sub < p.groups && before < p.topk_groups) kept[before] = sub;
      }
      wave_fence();
    }
    redo = redo || doubt;
    // the kept groups' values, four groups' reads ahead of their use
    for (int n = 0; n < p.topk_groups; n += 4) {
      int e0[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) e0[q] = kept[min(n + q, p.topk_groups - 1)] * size;
      const int cnt = p.topk_groups - n;
      if (quads) {
        for (int i = sub * 4; i < size; i += 4 * LPT) {
          float4 x[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<const float4*>(row + e0[q] + i);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < cnt) {
              list_insert<KL>(l, keys.of(x[q].x, e0[q] + i));
              list_insert<KL>(l, keys.of(x[q].y, e0[q] + i + 1));
              list_insert<KL>(l, keys.of(x[q].z, e0[q] + i + 2));
              list_insert<KL>(l, keys.of(x[q].w, e0[q] + i + 3));
            }
        }
      } else {
        for (int i = sub; i < size; i += LPT) {
          float x[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) x[q] = row[e0[q] + i];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < cnt) list_insert<KL>(l, keys.of(x[q], e0[q] + i));
        }
      }
    }
  }
  merge_round<1>(l);
  merge_round<2>(l);
  merge_round<4>(l);
  // Are the first k + 1 keys in order beyond doubt?  Part 0: masked, nothing is left
  // from there on, unless values lie below the window.
  const bool below = low < top - 0.9f * W;
  bool close = false, last = false;  // last: entries k - 1 and k
#pragma unroll
  for (int j = 0; j + 1 < KL; ++j) {
    const uint32_t a = l[j] >> 8, b = l[j + 1] >> 8;
    const bool tie = b != 0u && a - b <= near;
    if (j < p.k) {
      if (b == 0u && below) redo = true;
      close = close || tie;
    }
    if (j == p.k - 1) last = tie;
    if (j == p.k && last && (tie || (b == 0u && below))) redo = true;  // the list may end inside a run
  }
  // a softmax's c in 64 bits takes the sum over all experts: route_token
  if (close && p.bias && !p.sigmoid) redo = true;
  // lanes of a token with a doubtful lane: one bit a token
  uint64_t any = __ballot(redo && active);
  any |= any >> 4;
  any |= any >> 2;
  any |= any >> 1;
  any &= 0x0101010101010101ull;
  const bool skip = (any >> (tok * LPT)) & 1;
  // entry j = sub, sub + 8, .. of the list: its expert, its score from its logit
  // again, and its place
  constexpr int H = (KL + LPT - 1) / LPT;
  float s[H], cc[H];
  int id[H], at[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int j = sub + h * LPT;
    uint32_t key = 0u;
#pragma unroll
    for (int i = 0; i < KL; ++i) key = i == j ? l[i] : key;
    const bool some = (key >> 8) != 0u && j < KL && active;
    id[h] = some ? 255 - (int)(key & 255u) : -1;
    at[h] = j;
    const float x = some ? taken(zr[id[h]]) : -INFINITY;
    s[h] = some ? score(x) : 0.f;
    cc[h] = some ? s[h] + (p.bias ? p.bias[id[h]] : 0.f) : -INFINITY;
  }
  if (__any(close && active && !skip)) {  // not with a softmax and a bias
    // the listed experts in 64 bits
    double c[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const double x = id[h] >= 0 ? (double)taken(zr[id[h]]) : -INFINITY;
      c[h] = p.bias && id[h] >= 0 ? 1.0 / (1.0 + exp(-x)) + (double)taken(p.bias[id[h]]) : x;
      at[h] = 0;
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int n = 0; n < LPT; ++n) {
        const double oc = __shfl(c[h], tok * LPT + n, MOELB_WAVE);
        const int oi = __shfl(id[h], tok * LPT + n, MOELB_WAVE);
        const int oj = h * LPT + n;
#pragma unroll
        for (int g = 0; g < H; ++g)
          // entries without an expert keep their places behind the others
          at[g] += oi >= 0 ? (id[g] < 0 || oc > c[g] || (oc == c[g] && oi < id[g])) : (id[g] < 0 && oj < sub + g * LPT);
      }
  }
  float total = 0.f;
#pragma unroll
  for (int h = 0; h < H; ++h) total += at[h] < p.k ? s[h] : 0.f;
  total = token_all(total, add);
  // the scale last: over a sum of 0 it may be past the largest float
  const float share = p.renorm ? 1.0f / (total + 1e-20f) : 1.0f;
  float ck = 0.f, cn = 0.f;  // c of entries k - 1 and k
  bool more = false;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (at[h] < p.k && active && !skip) {
      p.idx[t * p.k + at[h]] = id[h];
      if (p.wts) p.wts[t * p.k + at[h]] = s[h] * share * p.scale;
    }
    ck += at[h] == p.k - 1 && id[h] >= 0 ? cc[h] : 0.f;
    cn += at[h] == p.k && id[h] >= 0 ? cc[h] : 0.f;
    more = more || (at[h] == p.k && id[h] >= 0);
  }
  if (p.gap) {
    // entries ranked in 64 bits may stand the other way round in fp32
    const float g = fmaxf(token_all(ck, add) - token_all(cn, add), 0.f);
    const float some = token_all(more ? 1.f : 0.f, add);
    if (sub == 0 && active && !skip) p.gap[t] = some > 0.f ? g : INFINITY;
  }
  return any;
}

template <int NV, int KL>
__global__ __launch_bounds__(WAVES * MOELB_WAVE) void route_kernel(RouteArgs p, int wave_floats) {
  extern __shared__ __align__(16) float smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* lds = smem + wave * wave_floats;
  const int t0 = (blockIdx.x * (blockDim.x >> 6) + wave) * TPW;
  if (t0 >= p.T) return;
  uint64_t todo = route_fast<NV, KL>(p, t0, lds);
  wave_fence();
#pragma unroll 1
  while (todo != 0ull) {
    const int tok = (__ffsll(static_cast<long long>(todo)) - 1) / LPT;
    todo &= todo - 1;
    double* cs = reinterpret_cast<double*>(lds);
    route_token(p, t0 + tok, cs, cs + p.E);
    wave_fence();
  }
}

template <int NV, int KL>
int launch_route(RouteArgs p, hipStream_t s) {
  // LDS of a wave: rows, group scores with their errors, and kept groups; the 64-bit form takes E +
  // groups doubles of it
  int floats = 0;
  if (p.groups > 1) {
    const int fast = TPW * (p.stride + 3 * p.groups), slow = 2 * (p.E + p.groups);
    floats = ((fast > slow ? fast : slow) + 3) / 4 * 4;
  }
  // few tokens: a wave a workgroup, so that they spread over the compute units
  const int per = p.T >= 4 * 256 * TPW ? WAVES : 1;
  const size_t lds = (size_t)per * floats * sizeof(float);
  if (!moelb_allow_lds(route_kernel<NV, KL>, lds)) return MOELB_ELAUNCH;
  constexpr int PART = 1 << 28;  // tokens a launch: its threads stay below 2^32
  for (int left = p.T; left > 0; left -= PART) {
    p.T = left < PART ? left : PART;
    const int blocks = (p.T + TPW * per - 1) / (TPW * per);
    hipLaunchKernelGGL((route_kernel<NV, KL>), dim3(blocks), dim3(per * MOELB_WAVE), lds, s, p, floats);
    MOELB_CHECK_LAUNCH();
    p.z += (size_t)p.T * p.E, p.idx += (size_t)p.T * p.k;
    if (p.wts) p.wts += (size_t)p.T * p.k;
    if (p.gap) p.gap += p.T;
  }
  return MOELB_OK;
}

template <int NV>
int launch_k(const RouteArgs& p, hipStream_t s) {
  if (p.k <= 2) return launch_route<NV, 4>(p, s);
  if (p.k <= 4) return launch_route<NV, 6>(p, s);
  if (p.k <= 8) return launch_route<NV, 10>(p, s);
  return launch_route<NV, 18>(p, s);
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
  const int vec = E % 4 == 0 && ((reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(bias)) & 15) == 0;
  const RouteArgs p = {z, bias, idx, wts, gap, T, E, k, score == MOELB_SCORE_SIGMOID, groups, topk_groups, group_top,
                       renorm != 0, scale, (E + 3) / 4 * 4 + 4, vec};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return E <= 32 ? launch_k<4>(p, s) : E <= 64 ? launch_k<8>(p, s) : E <= 128 ? launch_k<16>(p, s) : launch_k<32>(p, s);
}
