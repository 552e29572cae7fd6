// Gradients of the softmax router.
//
// Definition (FreeBalance, "FreeBalance: Pre-Routing Online MoE Load Balancing
// via Residual Workload Prediction", section 2.1 and eq. 4; the forward is
// moelb_gate_topk: the weight of a selected expert is its probability over all
// E).  With p = softmax(z), z = h W^T + b, and q_e the gradient that reaches
// expert e's weight (0 where e is not selected):
//   dz_e = p_e (q_e - S), S = sum_f p_f q_f
//   dh = dz W, dW = sum_t dz h[t]^T, db = sum_t dz
//
// Four steps on the tile of mfma_tile.h:
//   1. z (fp32), h and W both read along d
//   2. a wave per token: softmax, q from the token's k ids, dz in the storage
//      type (E padded to 64 with zeros), db partials per workgroup
//   3. dh = dz W (W read as columns, the sum runs over its rows) and dW = dz^T h
//      (both read as columns, the sum runs over tokens, cut into parts), one
//      launch
//   4. the parts of dW and db, added in order
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

__device__ __forceinline__ uint32_t bytes32(size_t n) { return n < mt::OUTSIDE ? (uint32_t)n : mt::OUTSIDE; }

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

__global__ __launch_bounds__(mt::THREADS) void gate_logits_f32_kernel(GateArgs<float> p) {
  __shared__ __align__(16) float lds[mt::S_FLOATS];
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  f32x16_t acc;
  auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.h + (size_t)(m0 + r) * p.d + k : nullptr; };
  auto pb = [&](int r, int k) { return n0 + r < p.E ? p.w + (size_t)(n0 + r) * p.d + k : nullptr; };
  mt::k_loop_f32<false, false>(lds, pa, pb, p.d, acc);
  mt::drain_f32<false>(lds, acc, [&](int r, int c, const float* v) {
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

__global__ __launch_bounds__(mt::THREADS) void gate_grads_kernel(GateArgs<uint16_t> p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  f32x16_t acc[GF][GF];
  if ((int)blockIdx.x < p.nh) {
    const int ntn = (p.d + GB - 1) / GB;
    const int m0 = blockIdx.x / ntn * GB, n0 = blockIdx.x % ntn * GB;
    mt::RowOp<GF> oa;
    mt::ColOp<GF, false> ob;
    oa.init(p.dz, bytes32((size_t)p.Ttok * p.Ep * 2), p.Ep, p.Ep, [&](int r) { return min(m0 + r, p.Ttok - 1); });
    ob.init(p.w, bytes32((size_t)p.E * p.d * 2), p.d, p.E, n0, p.d);
    mt::k_loop<GF, false>(lds, oa, ob, p.Ep / mt::BK, acc);
    mt::drain<GF, false>(lds, acc, [&](int r, int c, const float* v) { put_dh(p, m0 + r, n0 + c, v); });
    return;
  }
  int mi, ni, split, k0, n;
  dw_part(p, blockIdx.x - p.nh, GB, mi, ni, split, k0, n);
  mt::ColOp<GF, false> oa, ob;
  oa.init(p.dz + (size_t)k0 * p.Ep, bytes32((size_t)n * p.Ep * 2), p.Ep, n, mi * GB, p.Ep);
  ob.init(p.h + (size_t)k0 * p.d, bytes32((size_t)n * p.d * 2), p.d, n, ni * GB, p.d);
  mt::k_loop<GF, false>(lds, oa, ob, max(1, (n + mt::BK - 1) / mt::BK), acc);
  mt::drain<GF, false>(lds, acc, [&](int r, int c, const float* v) { put_dw(p, split, mi * GB + r, ni * GB + c, v); });
}

__global__ __launch_bounds__(mt::THREADS) void gate_grads_f32_kernel(GateArgs<float> p) {
  __shared__ __align__(16) float lds[mt::S_FLOATS];
  f32x16_t acc;
  if ((int)blockIdx.x < p.nh) {
    const int ntn = (p.d + 63) / 64;
    const int m0 = blockIdx.x / ntn * 64, n0 = blockIdx.x % ntn * 64;
    auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.dz + (size_t)(m0 + r) * p.Ep + k : nullptr; };
    auto pb = [&](int r, int k) { return n0 + r < p.d && k < p.E ? p.w + (size_t)k * p.d + n0 + r : nullptr; };
    mt::k_loop_f32<false, true>(lds, pa, pb, p.Ep, acc);
    mt::drain_f32<false>(lds, acc, [&](int r, int c, const float* v) { put_dh(p, m0 + r, n0 + c, v); });
    return;
  }
  int mi, ni, split, k0, n;
  dw_part(p, blockIdx.x - p.nh, 64, mi, ni, split, k0, n);
  const int m0 = mi * 64, n0 = ni * 64;
  auto pa = [&](int r, int k) { return m0 + r < p.Ep ? p.dz + (size_t)(k0 + k) * p.Ep + m0 + r : nullptr; };
  auto pb = [&](int r, int k) { return n0 + r < p.d ? p.h + (size_t)(k0 + k) * p.d + n0 + r : nullptr; };
  mt::k_loop_f32<true, true>(lds, pa, pb, n, acc);
  mt::drain_f32<false>(lds, acc, [&](int r, int c, const float* v) { put_dw(p, split, m0 + r, n0 + c, v); });
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
};
GateLayout gate_layout(int T, int d, int E, int dtype) {
  GateLayout l;
  const size_t eb = moelb_elem_bytes(dtype);
  l.Ep = (E + 63) & ~63;
  // step 2: 16 tokens a workgroup, at most 1024 of them
  l.blocks = (T + 15) / 16;
  l.blocks = l.blocks < 1 ? 1 : l.blocks > 1024 ? 1024 : l.blocks;
  // dW: parts of at least 256 tokens, enough for two workgroups a CU
  const int B = dtype == MOELB_BF16 ? GB : 64;
  const int tiles = ((d + B - 1) / B) * ((E + B - 1) / B);
  const int want = 512 / tiles, most = T / 256;
  l.splits = want < most ? want : most;
  l.splits = l.splits < 1 ? 1 : l.splits > 64 ? 64 : l.splits;
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

template <typename T>
int run(GateArgs<T> p, hipStream_t s) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int B = BF ? GB : 64;
  if constexpr (BF) {
    if (!moelb_allow_lds(gate_logits_kernel, mt::lds_bytes<GF>()) ||
        !moelb_allow_lds(gate_grads_kernel, mt::lds_bytes<GF>()))
      return MOELB_ELAUNCH;
  }
  if (p.Ttok > 0) {
    const dim3 grid((p.Ttok + B - 1) / B, (p.E + B - 1) / B);
    if constexpr (BF)
      hipLaunchKernelGGL(gate_logits_kernel, grid, dim3(mt::THREADS), mt::lds_bytes<GF>(), s, p);
    else
      hipLaunchKernelGGL(gate_logits_f32_kernel, grid, dim3(mt::THREADS), 0, s, p);
    MOELB_CHECK_LAUNCH();
  }
  const int st = launch_softmax(p, s);
  if (st != MOELB_OK) return st;
  const size_t ntn = (p.d + B - 1) / B;
  const size_t nh = p.dh && p.Ttok > 0 ? (size_t)((p.Ttok + B - 1) / B) * ntn : 0;
  const size_t nw = p.dw ? (size_t)((p.E + B - 1) / B) * ntn * p.splits : 0;
  if (nh + nw > 0x7fffffffull) return MOELB_EINVAL;
  p.nh = (int)nh;
  if (nh + nw > 0) {
    if constexpr (BF)
      hipLaunchKernelGGL(gate_grads_kernel, dim3((unsigned)(nh + nw)), dim3(mt::THREADS), mt::lds_bytes<GF>(), s, p);
    else
      hipLaunchKernelGGL(gate_grads_f32_kernel, dim3((unsigned)(nh + nw)), dim3(mt::THREADS), 0, s, p);
    MOELB_CHECK_LAUNCH();
  }
  const int sw = p.dw && p.splits > 1 ? (int)(((size_t)p.E * p.d / 8 + 255) / 256) : 0;
  const int sb = p.db ? (p.E + 3) / 4 : 0;
  if (sw + sb > 0) {
    hipLaunchKernelGGL((gate_sums_kernel<T>), dim3(sw + sb), dim3(256), 0, s, p, sw);
    MOELB_CHECK_LAUNCH();
  }
  return MOELB_OK;
}

}  // namespace

extern "C" size_t moelb_gate_backward_workspace_bytes(int T, int d, int E, int dtype) {
  if (T < 0 || d < 1 || E < 1 || E > MOELB_MAX_E || !moelb_dtype_ok(dtype)) return 0;
  return gate_layout(T, d, E, dtype).total;
}

extern "C" int moelb_gate_backward(const void* h, int T, int d, int E, int k, int dtype, const void* w, const float* b,
                                   const int32_t* idx, const float* dwts, void* ws, size_t ws_bytes, void* dh,
                                   void* dw, float* db, void* stream) {
  if (T < 0 || d <= 0 || d % 8 != 0 || E < 1 || E > MOELB_MAX_E || k < 1 || k > E || k > MOELB_MAX_K ||
      !moelb_dtype_ok(dtype))
    return MOELB_EINVAL;
  if (!w || !b || (T > 0 && (!h || !idx || !dwts))) return MOELB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(dh) |
       reinterpret_cast<uintptr_t>(dw)) & 15)
    return MOELB_EINVAL;
  const size_t eb = moelb_elem_bytes(dtype);
  if ((size_t)T * d * eb >= (1ull << 32) - 65536) return MOELB_EINVAL;
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
    return run<U>(p, static_cast<hipStream_t>(stream));
  };
  return dtype == MOELB_BF16 ? go(static_cast<uint16_t*>(nullptr)) : go(static_cast<float*>(nullptr));
}
