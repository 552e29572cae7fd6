// Logits of the current and the lookahead router, z = h W^T + b, in fp32.
//
// Definition: FreeBalance ("FreeBalance: Pre-Routing Online MoE Load Balancing
// via Residual Workload Prediction"), section 2.1 and eq. 2-4: the router that
// moelb_gate_topk fuses with its selection, here with the logits as the result.
//
// On the tile of mfma_tile.h: 128 tokens x 128 experts in bf16, 64 x 64 in fp32,
// a router after the other.
#include "mfma_tile.h"

namespace {

constexpr int LF = 2, LB = 64 * LF;  // 128 x 128 tiles

template <typename T>
struct LogitArgs {
  const T* h;
  const T* w[2];
  const float* b[2];
  float* z[2];
  int Ttok, d, E;
};

// 8 logits of row t from column c: the bias added, columns past E left out.
__device__ __forceinline__ void put_logits(float* z, const float* b, int E, size_t t, int c, const float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < E) z[t * E + c + i] = v[i] + (b ? b[c + i] : 0.f);
}

__global__ __launch_bounds__(mt::THREADS) void logits_kernel(LogitArgs<uint16_t> p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  const int m0 = blockIdx.x * LB, n0 = blockIdx.y * LB;
  const uint16_t* w = blockIdx.z ? p.w[1] : p.w[0];
  const float* b = blockIdx.z ? p.b[1] : p.b[0];
  float* z = blockIdx.z ? p.z[1] : p.z[0];
  mt::RowOp<LF> oa, ob;
  oa.init(p.h, (uint32_t)((size_t)p.Ttok * p.d * 2), p.d, p.d, [&](int r) { return min(m0 + r, p.Ttok - 1); });
  ob.init(w, (uint32_t)((size_t)p.E * p.d * 2), p.d, p.d, [&](int r) { return min(n0 + r, p.E - 1); });
  f32x16_t acc[LF][LF];
  mt::k_loop<LF, false>(lds, oa, ob, (p.d + mt::BK - 1) / mt::BK, acc);
  mt::drain<LF, false>(lds, acc, [&](int r, int c, const float* v) {
    if (m0 + r < p.Ttok) put_logits(z, b, p.E, m0 + r, n0 + c, v);
  });
}

__global__ __launch_bounds__(mt::S_THREADS) void logits_f32_kernel(LogitArgs<float> p) {
  __shared__ __align__(16) float lds[mt::STile<64>::FLOATS];
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  const float* w = blockIdx.z ? p.w[1] : p.w[0];
  const float* b = blockIdx.z ? p.b[1] : p.b[0];
  float* z = blockIdx.z ? p.z[1] : p.z[0];
  f32x16_t acc;
  auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.h + (size_t)(m0 + r) * p.d + k : nullptr; };
  auto pb = [&](int r, int k) { return n0 + r < p.E ? w + (size_t)(n0 + r) * p.d + k : nullptr; };
  mt::k_loop_f32<64, false, false>(lds, pa, pb, p.d, acc);
  mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) {
    if (m0 + r < p.Ttok) put_logits(z, b, p.E, m0 + r, n0 + c, v);
  });
}

int launch(const LogitArgs<uint16_t>& p, int routers, hipStream_t s) {
  if (!moelb_allow_lds(logits_kernel, mt::lds_bytes<LF>())) return MOELB_ELAUNCH;
  hipLaunchKernelGGL(logits_kernel, dim3((p.Ttok + LB - 1) / LB, (p.E + LB - 1) / LB, routers), dim3(mt::THREADS),
                     mt::lds_bytes<LF>(), s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}
int launch(const LogitArgs<float>& p, int routers, hipStream_t s) {
  hipLaunchKernelGGL(logits_f32_kernel, dim3((p.Ttok + 63) / 64, (p.E + 63) / 64, routers), dim3(mt::S_THREADS), 0, s,
                     p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

// Tokens in parts: the tile's operands are under mt::MAX_BYTES, a launch's
// threads under 2^32.
template <typename T>
int run_parts(LogitArgs<T> p, int T_all, int routers, hipStream_t s) {
  const size_t most = (mt::MAX_BYTES - 1) / ((size_t)p.d * sizeof(T));
  const int part = (int)(most < (1u << 24) ? (most > 128 ? most / 128 * 128 : most) : 1u << 24);
  for (long long t0 = 0; t0 < T_all; t0 += part) {
    LogitArgs<T> q = p;
    q.Ttok = (int)(T_all - t0 < part ? T_all - t0 : part);
    q.h += t0 * p.d;
    for (int r = 0; r < routers; ++r) q.z[r] += t0 * p.E;
    const int st = launch(q, routers, s);
    if (st != MOELB_OK) return st;
  }
  return MOELB_OK;
}

}  // namespace

extern "C" int moelb_gate_logits(const void* h, int T, int d, int E, int dtype, const void* w_cur, const float* b_cur,
                                 const void* w_next, const float* b_next, float* z, float* z_next, void* stream) {
  if (T < 0 || d <= 0 || d % 8 != 0 || d > 1 << 25 || E < 1 || E > MOELB_MAX_E || !moelb_dtype_ok(dtype))
    return MOELB_EINVAL;
  if (!w_cur || (!w_next && b_next)) return MOELB_EINVAL;
  if ((size_t)E * d * moelb_elem_bytes(dtype) >= mt::MAX_BYTES) return MOELB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(w_cur) | reinterpret_cast<uintptr_t>(w_next)) & 15)
    return MOELB_EINVAL;
  if (T == 0) return MOELB_OK;
  if (!h || !z || !w_next != !z_next) return MOELB_EINVAL;
  auto go = [&](auto* t) {
    using U = std::remove_pointer_t<decltype(t)>;
    LogitArgs<U> p = {static_cast<const U*>(h), {static_cast<const U*>(w_cur), static_cast<const U*>(w_next)},
                      {b_cur, b_next}, {z, z_next}, 0, d, E};
    return run_parts<U>(p, T, w_next ? 2 : 1, static_cast<hipStream_t>(stream));
  };
  return dtype == MOELB_BF16 ? go(static_cast<uint16_t*>(nullptr)) : go(static_cast<float*>(nullptr));
}
