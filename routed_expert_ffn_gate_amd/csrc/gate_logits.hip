// Logits of the current and the lookahead router, z = h W^T + b, in fp32.
//
// Definition: FreeBalance ("FreeBalance: Pre-Routing Online MoE Load Balancing
// via Residual Workload Prediction"), section 2.1 and eq. 2-4: the router that
// moelb_gate_topk fuses with its selection, here with the logits as the result.
//
// Many tokens: the tile of mfma_tile.h, 128 tokens x 128 experts in bf16, 64 x 64 in
// fp32; the tiles of the same tokens run side by side on one XCD, so its L2 serves
// h to all but the first.  Where the routers' experts fill 256 columns, a tile of 128 x
// 256 reads h once.  Few tokens: a tile of 16 x 16 by one workgroup, its waves
// taking the products' k in turn, so that a router's rows are read by E / 16 compute
// units at once.
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
  int nt;   // expert tiles of all routers
  int vec;  // rows of z start at 16 bytes
};

// 8 logits of row t from column c: the bias added, columns past E left out.
template <typename T>
__device__ __forceinline__ void put_logits(const LogitArgs<T>& p, float* z, const float* b, size_t t, int c,
                                           const float* v) {
  float* o = z + t * p.E + c;
  if (p.vec) {
#pragma unroll
    for (int h = 0; h < 8; h += 4)
      if (c + h < p.E) {
        float4 x = make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]);
        if (b) x.x += b[c + h], x.y += b[c + h + 1], x.z += b[c + h + 2], x.w += b[c + h + 3];
        *reinterpret_cast<float4*>(o + h) = x;
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < p.E) o[i] = v[i] + (b ? b[c + i] : 0.f);
}

// Workgroup b's token tile, router and expert tile: XCD b % 8 (workgroups go round)
// takes every eighth token tile, with all of its expert tiles in turn.
struct Where {
  int m, router, n;
};
template <typename T>
__device__ __forceinline__ Where where_of(const LogitArgs<T>& p, int b, int per_router) {
  const int j = b >> 3, n = j % p.nt;
  return {(j / p.nt) * 8 + (b & 7), n / per_router, n % per_router};
}

__global__ __launch_bounds__(mt::THREADS) void logits_kernel(LogitArgs<uint16_t> p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  const Where at = where_of(p, blockIdx.x, (p.E + LB - 1) / LB);
  const int m0 = at.m * LB, n0 = at.n * LB;
  if (m0 >= p.Ttok) return;
  const uint16_t* w = at.router ? p.w[1] : p.w[0];
  const float* b = at.router ? p.b[1] : p.b[0];
  float* z = at.router ? p.z[1] : p.z[0];
  mt::RowOp<LF> oa, ob;
  oa.init(p.h, (uint32_t)((size_t)p.Ttok * p.d * 2), p.d, p.d, [&](int r) { return min(m0 + r, p.Ttok - 1); });
  ob.init(w, (uint32_t)((size_t)p.E * p.d * 2), p.d, p.d, [&](int r) { return min(n0 + r, p.E - 1); });
  const int KT = (p.d + mt::BK - 1) / mt::BK;
  f32x16_t acc[LF][LF];
  mt::k_loop<LF, false>(lds, oa, ob, KT, acc, at.m % KT);
  mt::drain<LF, false>(lds, acc, [&](int r, int c, const float* v) {
    if (m0 + r < p.Ttok) put_logits(p, z, b, m0 + r, n0 + c, v);
  });
}

// Many tokens and 256 columns or 512, the experts of all routers side by side: eight
// waves take 128 tokens x 256 columns, so that h is read once for both routers of 128
// experts.  K steps of 64 go through a ring of three stages.  T = 32768, d = 4096, two
// routers of 128 experts 91 -> 83 us (3.7 TB/s), one of 256 86 -> 82; two of 256
// 160, either tile.  h further ahead than w (four to six stages, loaded by half of the
// waves) 84-97; h non-temporal 84-98.
constexpr int WM = 128, WN = 256, WAVES = 8, STAGES = 3;
constexpr int STAGE = (WM + WN) * 128;

__global__ __launch_bounds__(WAVES * MOELB_WAVE, 2) void logits_wide_kernel(LogitArgs<uint16_t> p) {
  constexpr int JA = WM / 8 / WAVES, JB = WN / 8 / WAVES, J = JA + JB;
  extern __shared__ __align__(16) char smem[];
  const int j8 = blockIdx.x >> 3, m0 = ((j8 / p.nt) * 8 + (blockIdx.x & 7)) * WM, n0 = j8 % p.nt * WN;
  if (m0 >= p.Ttok) return;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, fr = lane & 31, fh = lane >> 5;
  const int KT = (p.d + mt::BK - 1) / mt::BK, whole = p.d / mt::BK, turn = (m0 / WM) % KT;
  const uint32_t row = (uint32_t)p.d * 2u;
  // the wave loads weight rows of columns n0 + 32 wave .., all of one router
  const int c0 = n0 + wave * JB * 8;
  const mt::i32x4_t da = mt::descriptor(p.h, (uint32_t)p.Ttok * row);
  const mt::i32x4_t db = mt::descriptor(c0 < p.E ? p.w[0] : p.w[1], (uint32_t)p.E * row);
  uint32_t off[J], tail = 0;  // tail: in step `whole`, which instructions' chunks lie in K
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int r = j < JA ? (wave * JA + j) * 8 + (lane >> 3) : (wave * JB + j - JA) * 8 + (lane >> 3);
    const int c = mt::slot_of(r, lane & 7);
    const int from = j < JA ? min(m0 + r, p.Ttok - 1) : n0 + r - (c0 < p.E ? 0 : p.E);
    off[j] = (uint32_t)from * row + c * 16;
    tail |= (uint32_t)(c * 8 < p.d - whole * mt::BK) << j;
  }
  auto issue = [&](int t, int j) {
    const uint32_t st = lds0 + (uint32_t)(t % STAGES * STAGE);
    const int k = t + turn < KT ? t + turn : t + turn - KT;
    mt::copy16(k < whole || (tail >> j & 1) ? off[j] : mt::OUTSIDE, j < JA ? da : db, (uint32_t)k * 128u,
               st + (uint32_t)(j < JA ? (wave * JA + j) * 1024 : WM * 128 + (wave * JB + j - JA) * 1024));
  };
  int at[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) at[ks] = fr * 128 + mt::slot_of(fr, ks * 2 + fh) * 16;
  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i >> 1][i & 1][r] = 0.f;
  for (int t = 0; t < STAGES && t < KT; ++t)
#pragma unroll
    for (int j = 0; j < J; ++j) issue(t, j);
  mt::wait_stages<J, STAGES - 1>(min(STAGES, KT) - 1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  for (int t = 0; t < KT; ++t) {
    const char* sa = smem + t % STAGES * STAGE + wm * 64 * 128;
    const char* sb = smem + t % STAGES * STAGE + (WM + wn * 64) * 128;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) b[i] = *reinterpret_cast<const bf16x8_t*>(sb + i * 32 * 128 + at[ks]);
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] = *reinterpret_cast<const bf16x8_t*>(sa + i * 32 * 128 + at[ks]);
      if (ks == 3 && t + 1 < KT) {
        // lgkmcnt(0): this wave's reads of step t are done before its stage is refilled
        mt::wait_stages<J, STAGES - 2>(min(STAGES - 2, KT - 2 - t));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
#pragma unroll
      for (int mi = 0; mi < 2; ++mi) {
#pragma unroll
        for (int ni = 0; ni < 2; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[ni], a[mi], acc[mi][ni], 0, 0, 0);
        if (ks == 3 && t + STAGES < KT) {
#pragma unroll
          for (int j = mi; j < J; j += 2) issue(t + STAGES, j);
        }
      }
    }
  }
  __syncthreads();
  // The wave's 64 x 64 logits through LDS of its own, row r's 16-byte chunk c at c ^ (r
  // % 16), so that they leave in whole lines.
  char* o = smem + wave * 64 * 256;
#pragma unroll
  for (int mi = 0; mi < 2; ++mi)
#pragma unroll
    for (int ni = 0; ni < 2; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16_t& x = acc[mi][ni];
        *reinterpret_cast<float4*>(o + (mi * 32 + fr) * 256 + ((ni * 8 + q * 2 + fh) ^ (fr & 15)) * 16) =
            make_float4(x[q * 4], x[q * 4 + 1], x[q * 4 + 2], x[q * 4 + 3]);
      }
  const int v = n0 + wn * 64, r1 = v < p.E ? 0 : 1, c = v - r1 * p.E + (lane & 15) * 4;  // this lane's four columns
  const float* b = r1 ? p.b[1] : p.b[0];
  float* z = (r1 ? p.z[1] : p.z[0]) + c;
  float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
  if (b) add = make_float4(b[c], b[c + 1], b[c + 2], b[c + 3]);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = i * 4 + (lane >> 4), t = m0 + wm * 64 + r;
    float4 x = *reinterpret_cast<const float4*>(o + r * 256 + ((lane & 15) ^ (r & 15)) * 16);
    x.x += add.x, x.y += add.y, x.z += add.z, x.w += add.w;
    if (t < p.Ttok) *reinterpret_cast<float4*>(z + (size_t)t * p.E) = x;
  }
}

__global__ __launch_bounds__(mt::S_THREADS) void logits_f32_kernel(LogitArgs<float> p) {
  __shared__ __align__(16) float lds[mt::STile<64>::FLOATS];
  const Where at = where_of(p, blockIdx.x, (p.E + 63) / 64);
  const int m0 = at.m * 64, n0 = at.n * 64;
  if (m0 >= p.Ttok) return;
  const float* w = at.router ? p.w[1] : p.w[0];
  const float* b = at.router ? p.b[1] : p.b[0];
  float* z = at.router ? p.z[1] : p.z[0];
  f32x16_t acc;
  auto pa = [&](int r, int k) { return m0 + r < p.Ttok ? p.h + (size_t)(m0 + r) * p.d + k : nullptr; };
  auto pb = [&](int r, int k) { return n0 + r < p.E ? w + (size_t)(n0 + r) * p.d + k : nullptr; };
  mt::k_loop_f32<64, false, false>(lds, pa, pb, p.d, acc);
  mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) {
    if (m0 + r < p.Ttok) put_logits(p, z, b, m0 + r, n0 + c, v);
  });
}

// Few tokens.  A lane holds 16 bytes of a row: k (4 s + lane / 16) x 16 bytes of step
// s, token or expert lane % 16.  bf16: one v_mfma_f32_16x16x32_bf16 a step.  fp32: four
// v_mfma_f32_16x16x4_f32, the i-th with the i-th float of every lane (both operands
// take their k in the same order).  Wave w takes the steps w, w + FEW_WAVES, ..., four
// loads ahead of their use; the waves' sums are added in order.
constexpr int FEW_WAVES = 16;

template <typename T>
__global__ __launch_bounds__(FEW_WAVES * MOELB_WAVE) void logits_few_kernel(LogitArgs<T> p) {
  __shared__ float red[FEW_WAVES][256];
  constexpr int CH = 16 / (int)sizeof(T), AHEAD = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const T* w = blockIdx.z ? p.w[1] : p.w[0];
  const float* b = blockIdx.z ? p.b[1] : p.b[0];
  float* z = blockIdx.z ? p.z[1] : p.z[0];
  const int r = lane & 15, k0 = (lane >> 4) * CH;
  const T* hr = p.h + (size_t)min(t0 + r, p.Ttok - 1) * p.d;
  const T* wr = w + (size_t)min(e0 + r, p.E - 1) * p.d;
  const int steps = (p.d + 4 * CH - 1) / (4 * CH);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = wave; s0 < steps; s0 += FEW_WAVES * AHEAD) {
    uint4 x[AHEAD], y[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int k = (s0 + i * FEW_WAVES) * 4 * CH + k0;
      const bool in = k < p.d;  // d is a multiple of CH
      x[i] = in ? *reinterpret_cast<const uint4*>(hr + k) : make_uint4(0, 0, 0, 0);
      y[i] = in ? *reinterpret_cast<const uint4*>(wr + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if constexpr (sizeof(T) == 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x[i]),
                                                      __builtin_bit_cast(bf16x8_t, y[i]), acc, 0, 0, 0);
      } else {
        const f32x4_t u = __builtin_bit_cast(f32x4_t, x[i]), v = __builtin_bit_cast(f32x4_t, y[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(u[q], v[q], acc, 0, 0, 0);
      }
    }
  }
  *reinterpret_cast<f32x4_t*>(&red[wave][lane * 4]) = acc;  // token (lane / 16) * 4 + i, expert lane % 16
  __syncthreads();
  const int tok = threadIdx.x >> 4, e = threadIdx.x & 15;
  if (threadIdx.x < 256 && t0 + tok < p.Ttok && e0 + e < p.E) {
    float v = b ? b[e0 + e] : 0.f;
    const int at = ((tok >> 2) * 16 + e) * 4 + (tok & 3);
#pragma unroll
    for (int i = 0; i < FEW_WAVES; ++i) v += red[i][at];
    z[(size_t)(t0 + tok) * p.E + e0 + e] = v;
  }
}

// Whether a call runs faster in tiles of 16 x 16: up to about three of them a compute
// unit (fp32: six), where the large tiles would leave most units without work.  us,
// small | large tiles, bf16, both routers: 1 token, d = 4096, 128 experts 6.5 | 23.8;
// 512 tokens, d = 2048, 128 experts (512 tiles) 9.6 | 17.6; 1024 tokens, d = 4096, 128
// experts (1024) 31 | 28; 2048 tokens, d = 2048, 128 experts (2048) 31 | 18.  fp32:
// 1024 tokens, d = 4096, 128 experts 61 | 92; 2048 tokens, d = 2048, 128 experts 59 | 49.
template <typename T>
bool few_tokens(const LogitArgs<T>& p, int routers) {
  const size_t tiles = ((size_t)p.Ttok + 15) / 16 * ((p.E + 15) / 16) * routers;
  return tiles <= (sizeof(T) == 2 ? 768u : 1536u);
}

template <typename T>
int launch_few(const LogitArgs<T>& p, int routers, hipStream_t s) {
  hipLaunchKernelGGL((logits_few_kernel<T>), dim3((p.E + 15) / 16, (p.Ttok + 15) / 16, routers),
                     dim3(FEW_WAVES * MOELB_WAVE), 0, s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

// Whether a call takes the wide tile: no column of it is empty (two routers of 160
// experts 86 | 91, of 72, d = 1000, 37 | 40 us) and every compute unit gets one (T =
// 24576, d = 4096, two of 128, 62 | 63).
bool wide_columns(const LogitArgs<uint16_t>& p, int routers) {
  const int n = p.E * routers;
  return p.vec && n % WN == 0 && p.E % 128 == 0 && (size_t)(p.Ttok / WM) * (n / WN) >= 256;
}

int launch(LogitArgs<uint16_t> p, int routers, hipStream_t s) {
  if (wide_columns(p, routers)) {
    if (!moelb_allow_lds(logits_wide_kernel, STAGES * STAGE)) return MOELB_ELAUNCH;
    const int m = (p.Ttok + WM - 1) / WM;
    p.nt = p.E * routers / WN;
    hipLaunchKernelGGL(logits_wide_kernel, dim3((m + 7) / 8 * 8 * p.nt), dim3(WAVES * MOELB_WAVE), STAGES * STAGE, s,
                       p);
    MOELB_CHECK_LAUNCH();
    return MOELB_OK;
  }
  if (!moelb_allow_lds(logits_kernel, mt::lds_bytes<LF>())) return MOELB_ELAUNCH;
  const int m = (p.Ttok + LB - 1) / LB;
  p.nt = (p.E + LB - 1) / LB * routers;
  hipLaunchKernelGGL(logits_kernel, dim3((m + 7) / 8 * 8 * p.nt), dim3(mt::THREADS), mt::lds_bytes<LF>(), s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}
int launch(LogitArgs<float> p, int routers, hipStream_t s) {
  const int m = (p.Ttok + 63) / 64;
  p.nt = (p.E + 63) / 64 * routers;
  hipLaunchKernelGGL(logits_f32_kernel, dim3((m + 7) / 8 * 8 * p.nt), dim3(mt::S_THREADS), 0, s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

// Tokens in parts: the tile's operands are under mt::MAX_BYTES, a launch's
// threads under 2^32.
template <typename T>
int run_parts(LogitArgs<T> p, int T_all, int routers, hipStream_t s) {
  const size_t most = (mt::MAX_BYTES - 1) / ((size_t)p.d * sizeof(T));
  const int part = (int)(most < (1u << 22) ? (most > 128 ? most / 128 * 128 : most) : 1u << 22);
  for (long long t0 = 0; t0 < T_all; t0 += part) {
    LogitArgs<T> q = p;
    q.Ttok = (int)(T_all - t0 < part ? T_all - t0 : part);
    q.h += t0 * p.d;
    for (int r = 0; r < routers; ++r) q.z[r] += t0 * p.E;
    const int st = few_tokens(q, routers) ? launch_few(q, routers, s) : launch(q, routers, s);
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
                      {b_cur, b_next}, {z, z_next}, 0, d, E, 0, 0};
    p.vec = E % 4 == 0 && ((reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(z_next)) & 15) == 0;
    return run_parts<U>(p, T, w_next ? 2 : 1, static_cast<hipStream_t>(stream));
  };
  return dtype == MOELB_BF16 ? go(static_cast<uint16_t*>(nullptr)) : go(static_cast<float*>(nullptr));
}
