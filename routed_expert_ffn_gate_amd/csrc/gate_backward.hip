// Gradients of the softmax router, and of a router with another rule
// (moelb_route_backward, at the end: its dz, then the same products).
//
// Definition (FreeBalance, "FreeBalance: Pre-Routing Online MoE Load Balancing
// via Residual Workload Prediction", section 2.1 and eq. 4; the forward is
// moelb_gate_topk: the weight of a selected expert is its probability over all
// E).  With p = softmax(z), z = h W^T + b, and q_e the gradient that reaches
// expert e's weight (0 where e is not selected):
//   dz_e = p_e (q_e - S), S = sum_f p_f q_f
//   dh = dz W, dW = sum_t dz h[t]^T, db = sum_t dz
//
// On the tile of mfma_tile.h (bf16; fp32 on its fp32 tile):
//   1. z = h W^T, both read along d; up to 128 experts a tile holds whole rows
//      of z, so its epilogue goes on to dz and z never leaves LDS
//   2. dz: softmax, q from the token's k ids, dz in the storage type (E padded
//      to 64 with zeros), db partials per workgroup
//   3. dW = dz^T h (both read as columns, the sum runs over tokens, cut into
//      parts)
//   4. dh = dz W: a workgroup keeps its tokens' dz in registers and streams
//      tiles of W (read as columns) past them, storing as it goes; the bytes of
//      dh bound it
//   5. the parts of dW and db, added in order
//
// What bounds it: reading h twice (for z and for dW) and writing dh.  T = 32768,
// d = 4096, E = 128, bf16: step 1 and 2 in 77 us (3.5 TB/s of h), 3 and 4 in one
// launch of 135 us, 5 in 6 us.  Beyond 128 experts z and dz go through memory and
// W takes two buffers: E = 160 372 us, E = 256 386 (the call).  Small calls: three
// launches (T = 256, d = 256, E = 16, fp32: 10, 8 and 2 us).
#include <float.h>
#include <math.h>

#include "mfma_tile.h"

namespace {

constexpr int ROW_WAVES = 4;

template <typename T>
struct GateArgs {
  const T* h;
  const T* w;
  const float* b;
  const int32_t* idx;
  const float* dwts;
  float* z;     // [T][Ep]
  T* dz;        // [T][Ep]
  float* pdb;   // [blocks][Ep]
  float* pdw;   // [splits][E][d]
  T* dh;
  T* dw;
  float* db;
  int Ttok, d, E, Ep, k, splits, blocks, nh;  // nh: workgroups of dh in step 3
};

__device__ __forceinline__ uint32_t bytes32(size_t n) { return n < mt::MAX_BYTES ? (uint32_t)n : (uint32_t)mt::MAX_BYTES; }

// ---- 1: logits

constexpr int GF = 2;  // 128 x 128 tiles
constexpr int GB = 64 * GF;

__global__ __launch_bounds__(mt::THREADS) void gate_logits_kernel(GateArgs<uint16_t> p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  const int m0 = blockIdx.x * GB, n0 = blockIdx.y * GB;
  mt::RowOp<GF> oa, ob;
  oa.init(p.h, bytes32((size_t)p.Ttok * p.d * 2), p.d, p.d, [&](int r) { return min(m0 + r, p.Ttok - 1); });
  ob.init(p.w, bytes32((size_t)p.E * p.d * 2), p.d, p.d, [&](int r) { return min(n0 + r, p.E - 1); });
  f32x16_t acc[GF][GF];
  mt::k_loop<GF, false>(lds, oa, ob, (p.d + mt::BK - 1) / mt::BK, acc);
  mt::drain<GF, false>(lds, acc, [&](int r, int c, const float* v) {
    if (m0 + r < p.Ttok && n0 + c < p.Ep) mt::store8(p.z + (size_t)(m0 + r) * p.Ep + n0 + c, v);
  });
}

// All-reduce over 16 neighbouring lanes by row rotations.
template <class Op>
__device__ __forceinline__ float row_reduce(float v, Op op) {
  auto ror = [](float x, auto n) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x120 + decltype(n)::value, 0xf, 0xf, true));
  };
  v = op(v, ror(v, std::integral_constant<int, 8>{}));
  v = op(v, ror(v, std::integral_constant<int, 4>{}));
  v = op(v, ror(v, std::integral_constant<int, 2>{}));
  return op(v, ror(v, std::integral_constant<int, 1>{}));
}

// Steps 1 and 2 in one: the logits of ROWS tokens from m0 lie in LDS, get(r, c,
// v) reads NC of them; 16 lanes take a row, NC experts a lane, the workgroup
// THREADS / 16 rows at a time.  db partials to row blockIdx.x of pdb.  The
// caller has synchronised; `part` (THREADS NC floats) may be the logits' LDS.
// Picks: a lane's ids and gradients of all its rows, asked for before the logits
// are formed.
template <int N>
struct Picks {
  int id[N];
  float g[N];
};
template <typename T, int ROWS, int THREADS>
__device__ __forceinline__ void load_picks(const GateArgs<T>& p, int m0, Picks<ROWS * 16 / THREADS>& k) {
  const int s = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < ROWS * 16 / THREADS; ++i) {
    const int t = m0 + i * (THREADS / 16) + (threadIdx.x >> 4);
    const bool on = t < p.Ttok && s < p.k;
    k.id[i] = on ? p.idx[(size_t)t * p.k + s] : -1;
    k.g[i] = on ? p.dwts[(size_t)t * p.k + s] : 0.f;
  }
}
template <typename T, int NC, int ROWS, int THREADS, class Get>
__device__ __forceinline__ void softmax_rows(const GateArgs<T>& p, int m0, const Picks<ROWS * 16 / THREADS>& picks,
                                             float* part, Get get) {
  const int tid = threadIdx.x, lane = tid & 63, s = tid & 15, c = s * NC;
  auto add = [](float a, float b) { return a + b; };
  float bias[NC], db[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    bias[i] = c + i < p.E ? p.b[c + i] : 0.f;
    db[i] = 0.f;
  }
#pragma unroll
  for (int pass = 0; pass < ROWS * 16 / THREADS; ++pass) {
    const int r = pass * (THREADS / 16) + (tid >> 4), t = m0 + r;
    const bool on = t < p.Ttok;
    const int id = picks.id[pass];
    const float g = picks.g[pass];
    float z[NC], q[NC];
    float m = -INFINITY, sum = 0.f, pq = 0.f;
    get(r, c, z);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      z[i] = c + i < p.E ? z[i] + bias[i] : -INFINITY;
      m = fmaxf(m, z[i]);
      q[i] = 0.f;
    }
    m = row_reduce(m, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      z[i] = c + i < p.E ? (sizeof(T) == 2 ? __expf(z[i] - m) : expf(z[i] - m)) : 0.f;
      sum += z[i];
    }
    sum = 1.0f / row_reduce(sum, add);
    for (int j = 0; j < p.k; ++j) {
      const int e = __shfl(id, (lane & 48) + j, 64) - c;
      const float gj = __shfl(g, (lane & 48) + j, 64);
#pragma unroll
      for (int i = 0; i < NC; ++i) q[i] += e == i ? gj : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      z[i] *= sum;
      pq += z[i] * q[i];
    }
    pq = row_reduce(pq, add);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      z[i] = on && c + i < p.E ? z[i] * (q[i] - pq) : 0.f;
      db[i] += z[i];
    }
    // dz is rounded to the storage type: the matrix products that read it take
    // it beside h and w of that type
    if (on && c < p.Ep) {
      if constexpr (NC == 8)
        mt::store8(p.dz + (size_t)t * p.Ep + c, z);
      else
        *reinterpret_cast<float4*>(p.dz + (size_t)t * p.Ep + c) = make_float4(z[0], z[1], z[2], z[3]);
    }
  }
  // db: the lanes of an expert, added in order
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NC; ++i) part[(tid >> 4) * 16 * NC + c + i] = db[i];
  __syncthreads();
  if (tid < p.Ep) {
    float v = 0.f;
    for (int i = 0; i < THREADS / 16; ++i) v += part[i * 16 * NC + tid];
    p.pdb[(size_t)blockIdx.x * p.Ep + tid] = v;
  }
}

// E <= 128, bf16: 128 tokens a workgroup.
__global__ __launch_bounds__(mt::THREADS) void gate_dz_kernel(GateArgs<uint16_t> p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  const int m0 = blockIdx.x * GB;
  Picks<GB * 16 / mt::THREADS> picks;
  load_picks<uint16_t, GB, mt::THREADS>(p, m0, picks);
  {
    mt::RowOp<GF> oa, ob;
    oa.init(p.h, bytes32((size_t)p.Ttok * p.d * 2), p.d, p.d, [&](int r) { return min(m0 + r, p.Ttok - 1); });
    ob.init(p.w, bytes32((size_t)p.E * p.d * 2), p.d, p.d, [&](int r) { return min(r, p.E - 1); });
    const int KT = (p.d + mt::BK - 1) / mt::BK;
    f32x16_t acc[GF][GF];
    mt::k_loop<GF, false>(lds, oa, ob, KT, acc, blockIdx.x % KT);
    mt::stage<GF, false, 0>(lds, acc);
  }
  __syncthreads();
  float* st = reinterpret_cast<float*>(smem);
  softmax_rows<uint16_t, 8, GB, mt::THREADS>(p, m0, picks, st, [&](int r, int c, float* z) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(st + r * GB + ((c / 4 + h) ^ (r & 15)) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[h * 4 + i] = x[i];
    }
  });
}

// E <= 64, fp32: 64 tokens a workgroup.
__global__ __launch_bounds__(mt::S_THREADS) void gate_dz_f32_kernel(GateArgs<float> p) {
  __shared__ __align__(16) float lds[mt::STile<64>::FLOATS];
  const int m0 = blockIdx.x * 64;
  Picks<64 * 16 / mt::S_THREADS> picks;
  load_picks<float, 64, mt::S_THREADS>(p, m0, picks);
  f32x16_t acc;
  auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.h + (size_t)(m0 + r) * p.d + k : nullptr; };
  auto pb = [&](int r, int k) { return r < p.E ? p.w + (size_t)r * p.d + k : nullptr; };
  mt::k_loop_f32<64, false, false>(lds, pa, pb, p.d, acc);
  mt::stage_f32<64>(lds, acc);
  __syncthreads();
  softmax_rows<float, 4, 64, mt::S_THREADS>(p, m0, picks, lds, [&](int r, int c, float* z) {
    const f32x4_t x = mt::staged_f32<64>(lds, r, c / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = x[i];
  });
}

__global__ __launch_bounds__(mt::S_THREADS) void gate_logits_f32_kernel(GateArgs<float> p) {
  __shared__ __align__(16) float lds[mt::STile<64>::FLOATS];
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  f32x16_t acc;
  auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.h + (size_t)(m0 + r) * p.d + k : nullptr; };
  auto pb = [&](int r, int k) { return n0 + r < p.E ? p.w + (size_t)(n0 + r) * p.d + k : nullptr; };
  mt::k_loop_f32<64, false, false>(lds, pa, pb, p.d, acc);
  mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) {
    if (m0 + r < p.Ttok && n0 + c < p.Ep) mt::store8(p.z + (size_t)(m0 + r) * p.Ep + n0 + c, v);
  });
}

// ---- 2: softmax and its gradient

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, MOELB_WAVE));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, MOELB_WAVE);
  return v;
}

// Lane l of a wave holds experts l, l + 64, ...
template <typename T, int NE>
__global__ __launch_bounds__(MOELB_WAVE * ROW_WAVES) void gate_softmax_backward_kernel(GateArgs<T> p) {
  __shared__ float part[ROW_WAVES][NE * MOELB_WAVE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (p.Ttok + p.blocks - 1) / p.blocks;
  const int t0 = blockIdx.x * per, t1 = min(p.Ttok, t0 + per);
  float bias[NE], db[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + i * MOELB_WAVE;
    bias[i] = e < p.E ? p.b[e] : 0.f;
    db[i] = 0.f;
  }
  for (int t = t0 + wave; t < t1; t += ROW_WAVES) {
    float z[NE], q[NE];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + i * MOELB_WAVE;
      z[i] = e < p.E ? p.z[(size_t)t * p.Ep + e] + bias[i] : -INFINITY;
      q[i] = 0.f;
      m = fmaxf(m, z[i]);
    }
    const int id = lane < p.k ? p.idx[(size_t)t * p.k + lane] : -1;
    const float g = lane < p.k ? p.dwts[(size_t)t * p.k + lane] : 0.f;
    m = wave_max(m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + i * MOELB_WAVE;
      z[i] = e < p.E ? expf(z[i] - m) : 0.f;
      s += z[i];
    }
    s = 1.0f / wave_sum(s);
    for (int j = 0; j < p.k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), j));
#pragma unroll
      for (int i = 0; i < NE; ++i) q[i] += e == lane + i * MOELB_WAVE ? gj : 0.f;
    }
    float pq = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      z[i] *= s;
      pq += z[i] * q[i];
    }
    pq = wave_sum(pq);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + i * MOELB_WAVE;
      const float dz = e < p.E ? z[i] * (q[i] - pq) : 0.f;
      db[i] += dz;
      // rounded to the storage type: the matrix products below read it as an
      // operand, beside h and w of that type
      if (e < p.Ep) Elem<T>::store(p.dz, (size_t)t * p.Ep + e, dz);
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) part[wave][lane + i * MOELB_WAVE] = db[i];
  __syncthreads();
  for (int e = threadIdx.x; e < p.Ep; e += MOELB_WAVE * ROW_WAVES)
    p.pdb[(size_t)blockIdx.x * p.Ep + e] = (part[0][e] + part[1][e]) + (part[2][e] + part[3][e]);
}

// ---- the gradient of moelb_route's weights: dz from the kept logits
//
// With q_j the gradient of pick j's weight, s the scores and S = 1e-20 + the
// picks' sum of s:
//   ds_j = scale q_j, or scale (q_j - A / S) / S with A = sum_i q_i s_i (renorm)
//   sigmoid: dz = ds s (1 - s) at the picks; softmax: dz_e = s_e (ds_e - C), C =
//   sum_j s_j ds_j.  renorm: C = scale A 1e-20 / S^2, without the cancellation
//   of two sums that are equal but for the 1e-20.
// Computed from shares s / S, which a pick has in [0, 1], with the scale as the last
// factor: q / S alone may be past the largest float where the picks' scores vanish.
// 16 lanes take a token, lane s the experts s NC .. and pick s; sums go over the 16
// lanes by row rotations.  T = 32768, E = 128: 14 us (25 MB), where a wave a token
// with its chain of dependent loads took 22.
struct RouteRule {
  const float* z;  // [T][E]
  int sigmoid, renorm;
  float scale;
  int vec;  // rows of z start at 16 bytes
};

constexpr int DZ_THREADS = 256, DZ_ROWS = DZ_THREADS / 16;

template <typename T, int NC>
__global__ __launch_bounds__(DZ_THREADS) void route_dz_kernel(GateArgs<T> p, RouteRule u) {
  __shared__ float part[DZ_ROWS * 16 * NC];
  const int tid = threadIdx.x, lane = tid & 63, s = tid & 15, c = s * NC;
  auto add = [](float a, float b) { return a + b; };
  auto kept = [](float v) { return v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY; };  // masked: -inf and NaN
  float db[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) db[i] = 0.f;
  for (long long row0 = (long long)blockIdx.x * DZ_ROWS; row0 < p.Ttok; row0 += (long long)gridDim.x * DZ_ROWS) {
    const long long t = row0 + (tid >> 4);
    const bool on = t < p.Ttok;
    const float* zr = u.z + t * p.E;
    int id = on && s < p.k ? p.idx[t * p.k + s] : -1;
    if (id < 0 || id >= p.E) id = -1;
    const float q = id >= 0 ? p.dwts[t * p.k + s] : 0.f;
    float z[NC];  // softmax: this lane's experts' logits, then scores
    if (!u.sigmoid) {
#pragma unroll
      for (int i = 0; i < NC; i += 4) {
        if (u.vec) {
          float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          if (on && c + i < p.E) x = *reinterpret_cast<const float4*>(zr + c + i);
          z[i] = x.x, z[i + 1] = x.y, z[i + 2] = x.z, z[i + 3] = x.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) z[i + j] = on && c + i + j < p.E ? zr[c + i + j] : -INFINITY;
        }
      }
    }
    const float zj = id >= 0 ? kept(zr[id]) : -INFINITY;
    const bool live = zj > -INFINITY;
    float sj, cj;  // the pick's score, and 1 - s (sigmoid)
    if (u.sigmoid) {
      const float e = expf(-fabsf(zj)), r = 1.0f / (1.0f + e);
      sj = live ? (zj >= 0.f ? r : e * r) : 0.f;
      cj = zj >= 0.f ? e * r : r;
    } else {
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        z[i] = kept(z[i]);
        m = fmaxf(m, z[i]);
      }
      m = row_reduce(m, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        z[i] = z[i] > -INFINITY ? expf(z[i] - m) : 0.f;
        sum += z[i];
      }
      sum = row_reduce(sum, add);
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;  // 0: every logit is masked
#pragma unroll
      for (int i = 0; i < NC; ++i) z[i] *= inv;
      sj = live ? expf(zj - m) * inv : 0.f;
      cj = 0.f;
    }
    // dz = scale s r (hit - D), r = 1 / S (renorm) or 1
    const float r = u.renorm ? 1.0f / (row_reduce(sj, add) + 1e-20f) : 1.0f;
    const float share = sj * r, A = row_reduce(q * share, add);
    const float hit = id < 0 ? 0.f : u.renorm ? q - A : q, D = u.renorm ? A * 1e-20f : A;
    const float mine = u.sigmoid ? hit * share * cj : hit;
    float dz[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) dz[i] = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int e = __shfl(id, (lane & 48) + j, 64) - c;
      const float v = __shfl(mine, (lane & 48) + j, 64);
#pragma unroll
      for (int i = 0; i < NC; ++i) dz[i] += e == i ? v : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!u.sigmoid) dz[i] = z[i] * r * (dz[i] - D);
      dz[i] *= u.scale;
      db[i] += dz[i];
    }
    // rounded to the storage type: the matrix products below read it as an operand,
    // beside h and w of that type
    if (on) {
      T* o = p.dz + (size_t)t * p.Ep + c;
      if constexpr (NC % 8 == 0) {
#pragma unroll
        for (int i = 0; i < NC; i += 8) mt::store8(o + i, dz + i);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) Elem<T>::store(o, i, dz[i]);
      }
    }
  }
  // db: the tokens of an expert's lanes, added in order
#pragma unroll
  for (int i = 0; i < NC; ++i) part[(tid >> 4) * 16 * NC + c + i] = db[i];
  __syncthreads();
  for (int e = tid; e < p.Ep; e += DZ_THREADS) {
    float v = 0.f;
    for (int i = 0; i < DZ_ROWS; ++i) v += part[i * 16 * NC + e];
    p.pdb[(size_t)blockIdx.x * p.Ep + e] = v;
  }
}

// ---- 3: dh and dW

template <typename T>
__device__ __forceinline__ void put_dh(const GateArgs<T>& p, int t, int c, const float* v) {
  if (t < p.Ttok && c < p.d) mt::store8(p.dh + (size_t)t * p.d + c, v);
}
template <typename T>
__device__ __forceinline__ void put_dw(const GateArgs<T>& p, int split, int e, int c, const float* v) {
  if (e >= p.E || c >= p.d) return;
  const size_t at = (size_t)e * p.d + c;
  if (p.splits > 1)
    mt::store8(p.pdw + (size_t)split * p.E * p.d + at, v);
  else
    mt::store8(p.dw + at, v);
}
// Workgroup b of dW: its tokens [k0, k0 + n) and tile.
template <typename T>
__device__ __forceinline__ void dw_part(const GateArgs<T>& p, int b, int B, int& mi, int& ni, int& split, int& k0,
                                        int& n) {
  const int ntn = (p.d + B - 1) / B, ntm = (p.E + B - 1) / B;
  split = b / (ntm * ntn);
  b -= split * ntm * ntn;
  mi = b / ntn;
  ni = b % ntn;
  const int steps = (p.Ttok + 63) / 64, ps = (steps + p.splits - 1) / p.splits * 64;
  k0 = min(p.Ttok, split * ps);
  n = min(p.Ttok, k0 + ps) - k0;
}

__device__ __forceinline__ void dw_tile(const GateArgs<uint16_t>& p, int block, uint16_t* lds) {
  f32x16_t acc[GF][GF];
  int mi, ni, split, k0, n;
  dw_part(p, block, GB, mi, ni, split, k0, n);
  mt::ColOp<GF, false> oa, ob;
  oa.init(p.dz + (size_t)k0 * p.Ep, bytes32((size_t)n * p.Ep * 2), p.Ep, n, mi * GB, p.Ep);
  ob.init(p.h + (size_t)k0 * p.d, bytes32((size_t)n * p.d * 2), p.d, n, ni * GB, p.d);
  mt::k_loop<GF, false>(lds, oa, ob, max(1, (n + mt::BK - 1) / mt::BK), acc);
  mt::drain<GF, false>(lds, acc, [&](int r, int c, const float* v) { put_dw(p, split, mi * GB + r, ni * GB + c, v); });
}

// dh for 128 tokens and every parts-th 128-column tile from `part` on.  Wave
// (wm, wn): 64 tokens, whose dz it keeps as fragments, x 64 columns.  A tile of
// W (Ep rows x 128 columns, KB half-stages) is loaded NBUF - 1 tiles ahead.
// With three buffers the wait at a tile's use lets as many later operations be
// outstanding as one tile has loads: later are at least those, so the tile
// itself has landed, however many stores lie between.  The two lane halves
// trade 4-column runs, so that a lane stores 8 adjacent columns of its token.
template <int KB>
constexpr int dh_buffers() { return KB == 1 ? 3 : 2; }

template <int KB>
__device__ __forceinline__ void dh_tiles(const GateArgs<uint16_t>& p, int mi_, int part, int parts, uint16_t* lds) {
  constexpr int NBUF = dh_buffers<KB>();
  constexpr int HALF = mt::half_elems<GF>(), TILE = KB * HALF, NI = 2 * GF;
  const uint32_t lds_u32 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fh = lane >> 5;
  const int m0 = mi_ * GB + wm * 64;
  const int ntn = (p.d + GB - 1) / GB, n = (ntn - part + parts - 1) / parts;
  const uint32_t bytes = bytes32((size_t)p.E * p.d * 2);
  // the tiles in turn, each workgroup from another one on (the same columns of
  // rows 4 KiB apart lie on one memory channel)
  auto col = [&](int i) { return (part + (i + mi_) % n * parts) * GB; };
  auto issue = [&](int i) {
    mt::ColOp<GF, false> ob;
    ob.init(p.w, bytes, p.d, p.E, col(i), p.d);
#pragma unroll
    for (int h = 0; h < KB; ++h)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        ob.issue(h, j, lds_u32 + (uint32_t)((i % NBUF) * TILE + h * HALF + (wave * NI + j) * 512) * 2u);
  };
  bf16x8_t fa[2][KB * 4];
#pragma unroll
  for (int mi = 0; mi < 2; ++mi) {
    const uint16_t* row = p.dz + (size_t)min(m0 + mi * 32 + fr, p.Ttok - 1) * p.Ep + fh * 8;
#pragma unroll
    for (int k = 0; k < KB * 4; ++k) fa[mi][k] = *reinterpret_cast<const bf16x8_t*>(row + k * 16);
  }
#pragma unroll
  for (int mi = 0; mi < 2; ++mi)
#pragma unroll
    for (int k = 0; k < KB * 4; ++k) asm volatile("" : "+v"(fa[mi][k]));  // landed before the first DMA
  mt::FragAt<GF, true> fb;
  fb.init(wn, 0);
  for (int i = 0; i < NBUF - 1 && i < n; ++i) issue(i);
  for (int i = 0; i < n; ++i) {
    if (NBUF == 3 && i + 1 < n)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(KB * NI) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (i + NBUF - 1 < n) issue(i + NBUF - 1);
    f32x16_t acc[2][2];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int ni = 0; ni < 2; ++ni)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[mi][ni][q] = 0.f;
#pragma unroll
    for (int h = 0; h < KB; ++h) {
      const uint16_t* half = lds + (i % NBUF) * TILE + h * HALF;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int ni = 0; ni < 2; ++ni) {
          const bf16x8_t f = fb.read(half, k, ni, 0);
#pragma unroll
          for (int mi = 0; mi < 2; ++mi)
            acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, fa[mi][h * 4 + k], acc[mi][ni], 0, 0, 0);
        }
    }
    const int c0 = col(i) + wn * 64 + fh * 8;
#pragma unroll
    for (int mi = 0; mi < 2; ++mi) {
      const int t = m0 + mi * 32 + fr;
      uint16_t* o = p.dh + (size_t)min(t, p.Ttok - 1) * p.d + c0;
#pragma unroll
      for (int ni = 0; ni < 2; ++ni)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const f32x16_t& a = acc[mi][ni];
          uint32_t x0 = bf16x2_pack(a[q * 4], a[q * 4 + 1]), x1 = bf16x2_pack(a[q * 4 + 2], a[q * 4 + 3]);
          uint32_t y0 = bf16x2_pack(a[q * 4 + 4], a[q * 4 + 5]), y1 = bf16x2_pack(a[q * 4 + 6], a[q * 4 + 7]);
          // lane halves: columns 8q + 0..3 | 4..7 and 8q + 8..11 | 12..15
          const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
          const int c = ni * 32 + q * 8;
          if (t < p.Ttok && c0 + c < p.d)
            *reinterpret_cast<uint4*>(o + c) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
        }
    }
  }
}

// dW and dh in one launch, their workgroups spread evenly over it: one reads h,
// the other writes dh.
template <int KB>
__global__ __launch_bounds__(mt::THREADS) void gate_grads_kernel(GateArgs<uint16_t> p, int parts) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  const long long b = blockIdx.x, total = gridDim.x;
  const int before = (int)(b * p.nh / total);  // dh workgroups before this one
  if ((b + 1) * p.nh / total > before)
    dh_tiles<KB>(p, before / parts, before % parts, parts, lds);
  else
    dw_tile(p, (int)b - before, lds);
}

__global__ __launch_bounds__(mt::S_THREADS) void gate_grads_f32_kernel(GateArgs<float> p) {
  __shared__ __align__(16) float lds[mt::STile<64>::FLOATS];
  f32x16_t acc;
  if ((int)blockIdx.x < p.nh) {
    const int ntn = (p.d + 63) / 64;
    const int m0 = blockIdx.x / ntn * 64, n0 = blockIdx.x % ntn * 64;
    auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.dz + (size_t)(m0 + r) * p.Ep + k : nullptr; };
    auto pb = [&](int r, int k) { return n0 + r < p.d && k < p.E ? p.w + (size_t)k * p.d + n0 + r : nullptr; };
    mt::k_loop_f32<64, false, true>(lds, pa, pb, p.Ep, acc);
    mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) { put_dh(p, m0 + r, n0 + c, v); });
    return;
  }
  int mi, ni, split, k0, n;
  dw_part(p, blockIdx.x - p.nh, 64, mi, ni, split, k0, n);
  const int m0 = mi * 64, n0 = ni * 64;
  auto pa = [&](int r, int k) { return m0 + r < p.Ep ? p.dz + (size_t)(k0 + k) * p.Ep + m0 + r : nullptr; };
  auto pb = [&](int r, int k) { return n0 + r < p.d ? p.h + (size_t)(k0 + k) * p.d + n0 + r : nullptr; };
  mt::k_loop_f32<64, true, true>(lds, pa, pb, n, acc);
  mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) { put_dw(p, split, m0 + r, n0 + c, v); });
}

// ---- 4: sums over the parts.  Blocks below nw: dW, 8 values a thread; the
// rest: a wave per expert adds the db partials (lanes strided, then a fixed
// tree).
template <typename T>
__global__ __launch_bounds__(256) void gate_sums_kernel(GateArgs<T> p, int nw) {
  if ((int)blockIdx.x < nw) {
    const size_t n8 = (size_t)p.E * p.d / 8, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    float v[8];
    mt::load8(p.pdw + i * 8, v);
#pragma unroll 8
    for (int s = 1; s < p.splits; ++s) {
      float u[8];
      mt::load8(p.pdw + ((size_t)s * n8 + i) * 8, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    mt::store8(p.dw + i * 8, v);
    return;
  }
  const int e = (blockIdx.x - nw) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (e >= p.E) return;
  float v = 0.f;
  for (int i = lane; i < p.blocks; i += MOELB_WAVE) v += p.pdb[(size_t)i * p.Ep + e];
  v = wave_sum(v);
  if (lane == 0) p.db[e] = v;
}

// ---- host

struct GateLayout {
  size_t z, dz, pdb, pdw, total;
  int Ep, blocks, splits;
  bool fused;
};
GateLayout gate_layout(int T, int d, int E, int dtype) {
  GateLayout l;
  const size_t eb = moelb_elem_bytes(dtype);
  l.Ep = (E + 63) & ~63;
  // db partials: one a tile (bf16: 128 tokens, E <= 128; fp32: 64, 64), else a token a
  // wave, at most 1024 workgroups
  const int tok = dtype == MOELB_BF16 ? GB : 64;
  l.fused = l.Ep <= tok;
  l.blocks = l.fused ? (T + tok - 1) / tok : (T + 3) / 4;
  l.blocks = l.blocks < 1 ? 1 : !l.fused && l.blocks > 1024 ? 1024 : l.blocks;
  // dW: parts of at least 256 tokens, about a workgroup a compute unit (twice as
  // many: 245 against 212 us at T = 32768, d = 4096, E = 128)
  const int B = dtype == MOELB_BF16 ? GB : 64;
  const int tiles = ((d + B - 1) / B) * ((E + B - 1) / B);
  const int want = 256 / tiles, most = T / 256;
  l.splits = want < most ? want : most;
  l.splits = l.splits < 1 ? 1 : l.splits > 16 ? 16 : l.splits;
  l.z = 0;
  l.dz = moelb_align256((size_t)T * l.Ep * 4);
  l.pdb = l.dz + moelb_align256((size_t)T * l.Ep * eb);
  l.pdw = l.pdb + moelb_align256((size_t)l.blocks * l.Ep * 4);
  l.total = l.pdw + (l.splits > 1 ? moelb_align256((size_t)l.splits * E * d * 4) : 0);
  return l;
}

template <typename T>
int launch_softmax(const GateArgs<T>& p, hipStream_t s) {
  const dim3 grid(p.blocks), wg(MOELB_WAVE * ROW_WAVES);
  switch (p.Ep / 64) {
    case 1:
      hipLaunchKernelGGL((gate_softmax_backward_kernel<T, 1>), grid, wg, 0, s, p);
      break;
    case 2:
      hipLaunchKernelGGL((gate_softmax_backward_kernel<T, 2>), grid, wg, 0, s, p);
      break;
    case 3:
      hipLaunchKernelGGL((gate_softmax_backward_kernel<T, 3>), grid, wg, 0, s, p);
      break;
    default:
      hipLaunchKernelGGL((gate_softmax_backward_kernel<T, 4>), grid, wg, 0, s, p);
  }
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

template <int KB>
int launch_grads(GateArgs<uint16_t> p, hipStream_t s) {
  constexpr size_t dh = (size_t)dh_buffers<KB>() * KB * mt::half_elems<GF>() * sizeof(uint16_t);
  constexpr size_t lds = dh > mt::lds_bytes<GF>() ? dh : mt::lds_bytes<GF>();
  if (!moelb_allow_lds(gate_grads_kernel<KB>, lds)) return MOELB_ELAUNCH;
  const int m = (p.Ttok + GB - 1) / GB, ntn = (p.d + GB - 1) / GB;
  // dh: about a workgroup a compute unit where there are few tokens
  int parts = m > 0 ? (256 + m - 1) / m : 1;
  if (parts > ntn) parts = ntn;
  p.nh = p.dh ? m * parts : 0;
  const int nw = p.dw ? ((p.E + GB - 1) / GB) * ntn * p.splits : 0;
  if (p.nh + nw == 0) return MOELB_OK;
  hipLaunchKernelGGL((gate_grads_kernel<KB>), dim3(p.nh + nw), dim3(mt::THREADS), lds, s, p, parts);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

int run_dz(const GateArgs<uint16_t>& p, bool fused, hipStream_t s) {
  constexpr size_t lds = mt::lds_bytes<GF>();
  if (p.Ttok > 0 && fused) {
    if (!moelb_allow_lds(gate_dz_kernel, lds)) return MOELB_ELAUNCH;
    hipLaunchKernelGGL(gate_dz_kernel, dim3(p.blocks), dim3(mt::THREADS), lds, s, p);
    MOELB_CHECK_LAUNCH();
  } else {
    if (p.Ttok > 0) {
      if (!moelb_allow_lds(gate_logits_kernel, lds)) return MOELB_ELAUNCH;
      hipLaunchKernelGGL(gate_logits_kernel, dim3((p.Ttok + GB - 1) / GB, (p.E + GB - 1) / GB), dim3(mt::THREADS), lds,
                         s, p);
      MOELB_CHECK_LAUNCH();
    }
    const int st = launch_softmax(p, s);
    if (st != MOELB_OK) return st;
  }
  return MOELB_OK;
}

int run_grads(const GateArgs<uint16_t>& p, hipStream_t s) {
  switch (p.Ep / 64) {
    case 1:
      return launch_grads<1>(p, s);
    case 2:
      return launch_grads<2>(p, s);
    case 3:
      return launch_grads<3>(p, s);
    default:
      return launch_grads<4>(p, s);
  }
}

// Workgroups of dh and of dW in fp32.
void grads_grid(const GateArgs<float>& p, size_t& nh, size_t& nw) {
  const size_t ntn = (p.d + 63) / 64;
  nh = p.dh ? (size_t)((p.Ttok + 63) / 64) * ntn : 0;
  nw = p.dw ? (size_t)((p.E + 63) / 64) * ntn * p.splits : 0;
}
bool launches_ok(const GateArgs<float>& p) {
  size_t nh, nw;
  grads_grid(p, nh, nw);
  return nh + nw <= moelb_most_blocks(mt::S_THREADS);
}
// bf16 rows are at most 2^25 elements, T d and E d below 2^31 of them: T / 128 x
// d / 128 workgroups of 256 threads and less
bool launches_ok(const GateArgs<uint16_t>&) { return true; }

int run_dz(const GateArgs<float>& p, bool fused, hipStream_t s) {
  if (fused) {
    hipLaunchKernelGGL(gate_dz_f32_kernel, dim3(p.blocks), dim3(mt::S_THREADS), 0, s, p);
    MOELB_CHECK_LAUNCH();
  } else {
    if (p.Ttok > 0) {
      hipLaunchKernelGGL(gate_logits_f32_kernel, dim3((p.Ttok + 63) / 64, (p.E + 63) / 64), dim3(mt::S_THREADS), 0, s,
                         p);
      MOELB_CHECK_LAUNCH();
    }
    const int st = launch_softmax(p, s);
    if (st != MOELB_OK) return st;
  }
  return MOELB_OK;
}

int run_grads(GateArgs<float> p, hipStream_t s) {
  size_t nh, nw;
  grads_grid(p, nh, nw);
  p.nh = (int)nh;
  if (nh + nw > 0) {
    hipLaunchKernelGGL(gate_grads_f32_kernel, dim3((unsigned)(nh + nw)), dim3(mt::S_THREADS), 0, s, p);
    MOELB_CHECK_LAUNCH();
  }
  return MOELB_OK;
}

// The products from dz, and the sums over their parts.
template <typename T>
int run_products(const GateArgs<T>& p, hipStream_t s) {
  const int st = run_grads(p, s);
  if (st != MOELB_OK) return st;
  const int sw = p.dw && p.splits > 1 ? (int)(((size_t)p.E * p.d / 8 + 255) / 256) : 0;
  const int sb = p.db ? (p.E + 3) / 4 : 0;
  if (sw + sb > 0) {
    hipLaunchKernelGGL((gate_sums_kernel<T>), dim3(sw + sb), dim3(256), 0, s, p, sw);
    MOELB_CHECK_LAUNCH();
  }
  return MOELB_OK;
}

template <typename T>
int run_all(const GateArgs<T>& p, bool fused, hipStream_t s) {
  const int st = run_dz(p, fused, s);
  return st != MOELB_OK ? st : run_products(p, s);
}

// moelb_route_backward: dz from the caller's logits, then the products.
template <typename T>
int run_route(const GateArgs<T>& p, const RouteRule& u, hipStream_t s) {
  const dim3 grid(p.blocks), wg(DZ_THREADS);
  switch (p.Ep / 64) {  // NC = Ep / 16 experts a lane
    case 1:
      hipLaunchKernelGGL((route_dz_kernel<T, 4>), grid, wg, 0, s, p, u);
      break;
    case 2:
      hipLaunchKernelGGL((route_dz_kernel<T, 8>), grid, wg, 0, s, p, u);
      break;
    case 3:
      hipLaunchKernelGGL((route_dz_kernel<T, 12>), grid, wg, 0, s, p, u);
      break;
    default:
      hipLaunchKernelGGL((route_dz_kernel<T, 16>), grid, wg, 0, s, p, u);
  }
  MOELB_CHECK_LAUNCH();
  return run_products(p, s);
}

// The route's layout: as the softmax router's, without z, and dz by 16 tokens a
// workgroup at any E.
GateLayout route_layout(int T, int d, int E, int dtype) {
  GateLayout l = gate_layout(T, d, E, dtype);
  const int blocks = (int)(((size_t)T + DZ_ROWS - 1) / DZ_ROWS);
  l.blocks = blocks < 1 ? 1 : blocks > 512 ? 512 : blocks;
  const size_t pdw = l.total - l.pdw;
  l.dz = 0;
  l.pdb = moelb_align256((size_t)T * l.Ep * moelb_elem_bytes(dtype));
  l.pdw = l.pdb + moelb_align256((size_t)l.blocks * l.Ep * 4);
  l.total = l.pdw + pdw;
  return l;
}

// What both entry points require of sizes, operands and outputs.
bool backward_args_ok(const void* h, int T, int d, int E, int k, int dtype, const void* w, const int32_t* idx,
                      const float* dwts, const void* dh, const void* dw) {
  if (T < 0 || d <= 0 || d % 8 != 0 || E < 1 || E > MOELB_MAX_E || k < 1 || k > E || k > MOELB_MAX_K ||
      !moelb_dtype_ok(dtype))
    return false;
  if (!w || (T > 0 && (!h || !idx || !dwts))) return false;
  if ((reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(dh) |
       reinterpret_cast<uintptr_t>(dw)) & 15)
    return false;
  const size_t eb = moelb_elem_bytes(dtype);
  // a column operand's 64 rows of a step, those past the last included, have
  // 32-bit offsets
  if (dtype == MOELB_BF16 && d > 1 << 25) return false;
  // h, w and dz are operands of the tile
  const size_t Ep = ((size_t)E + 63) / 64 * 64, most = mt::MAX_BYTES;
  return (size_t)T * d * eb < most && (size_t)E * d * eb < most && (size_t)T * Ep * eb < most;
}

}  // namespace

extern "C" size_t moelb_gate_backward_workspace_bytes(int T, int d, int E, int dtype) {
  if (T < 0 || d < 1 || E < 1 || E > MOELB_MAX_E || !moelb_dtype_ok(dtype)) return 0;
  return gate_layout(T, d, E, dtype).total;
}

extern "C" int moelb_gate_backward(const void* h, int T, int d, int E, int k, int dtype, const void* w, const float* b,
                                   const int32_t* idx, const float* dwts, void* ws, size_t ws_bytes, void* dh,
                                   void* dw, float* db, void* stream) {
  if (!backward_args_ok(h, T, d, E, k, dtype, w, idx, dwts, dh, dw) || !b) return MOELB_EINVAL;
  const GateLayout l = gate_layout(T, d, E, dtype);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < l.total) return MOELB_EWORKSPACE;
  if (!dh && !dw && !db) return MOELB_OK;
  char* base = static_cast<char*>(ws);
  auto go = [&](auto* t) {
    using U = std::remove_pointer_t<decltype(t)>;
    GateArgs<U> p = {};
    p.h = static_cast<const U*>(h);
    p.w = static_cast<const U*>(w);
    p.b = b, p.idx = idx, p.dwts = dwts;
    p.z = reinterpret_cast<float*>(base + l.z);
    p.dz = reinterpret_cast<U*>(base + l.dz);
    p.pdb = reinterpret_cast<float*>(base + l.pdb);
    p.pdw = reinterpret_cast<float*>(base + l.pdw);
    p.dh = static_cast<U*>(dh);
    p.dw = static_cast<U*>(dw);
    p.db = db;
    p.Ttok = T, p.d = d, p.E = E, p.Ep = l.Ep, p.k = k, p.splits = l.splits, p.blocks = l.blocks;
    if (!launches_ok(p)) return (int)MOELB_EINVAL;
    return run_all<U>(p, l.fused && T > 0, static_cast<hipStream_t>(stream));
  };
  return dtype == MOELB_BF16 ? go(static_cast<uint16_t*>(nullptr)) : go(static_cast<float*>(nullptr));
}

extern "C" size_t moelb_route_backward_workspace_bytes(int T, int d, int E, int dtype) {
  if (T < 0 || d < 1 || E < 1 || E > MOELB_MAX_E || !moelb_dtype_ok(dtype)) return 0;
  return route_layout(T, d, E, dtype).total;
}

extern "C" int moelb_route_backward(const void* h, int T, int d, int E, int k, int dtype, const void* w, const float* z,
                                    const int32_t* idx, const float* dwts, int score, int renorm, float scale, void* ws,
                                    size_t ws_bytes, void* dh, void* dw, float* db, void* stream) {
  if (!backward_args_ok(h, T, d, E, k, dtype, w, idx, dwts, dh, dw) || (T > 0 && !z)) return MOELB_EINVAL;
  if (score != MOELB_SCORE_SOFTMAX && score != MOELB_SCORE_SIGMOID) return MOELB_EINVAL;
  if (!(fabsf(scale) <= FLT_MAX)) return MOELB_EINVAL;
  const GateLayout l = route_layout(T, d, E, dtype);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < l.total) return MOELB_EWORKSPACE;
  if (!dh && !dw && !db) return MOELB_OK;
  char* base = static_cast<char*>(ws);
  auto go = [&](auto* t) {
    using U = std::remove_pointer_t<decltype(t)>;
    GateArgs<U> p = {};
    p.h = static_cast<const U*>(h);
    p.w = static_cast<const U*>(w);
    p.idx = idx, p.dwts = dwts;
    p.dz = reinterpret_cast<U*>(base + l.dz);
    p.pdb = reinterpret_cast<float*>(base + l.pdb);
    p.pdw = reinterpret_cast<float*>(base + l.pdw);
    p.dh = static_cast<U*>(dh);
    p.dw = static_cast<U*>(dw);
    p.db = db;
    p.Ttok = T, p.d = d, p.E = E, p.Ep = l.Ep, p.k = k, p.splits = l.splits, p.blocks = l.blocks;
    if (!launches_ok(p)) return (int)MOELB_EINVAL;
    const RouteRule u = {z, score == MOELB_SCORE_SIGMOID, renorm != 0, scale,
                         E % 4 == 0 && (reinterpret_cast<uintptr_t>(z) & 15) == 0};
    return run_route<U>(p, u, static_cast<hipStream_t>(stream));
  };
  return dtype == MOELB_BF16 ? go(static_cast<uint16_t*>(nullptr)) : go(static_cast<float*>(nullptr));
}
