// Experts in microscaled 4-bit floating point: quantisation, reading back, and
// the grouped FFN on tokens, activations and weights in that format.
//
// Definition (include/moelb.h, moelb_mx_quantize and moelb_mx_grouped_ffn): the
// OCP MX format with e2m1 elements; the FFN is moelb_grouped_ffn's (FreeBalance,
// "FreeBalance: Pre-Routing Online MoE Load Balancing via Residual Workload
// Prediction", section 2.1) with both factors of every product in it.
//
// One wave per 32 x 32 block of an expert's rows and columns, its fragments
// straight from memory, v_mfma_scale_f32_32x32x64_f8f6f4.  The weights'
// fragment is the instruction's first operand, so a lane ends with 16 columns
// of one row: the block's magnitude, codes and scale are formed between two
// lanes, without LDS.
#include "ffn_sched.h"
#include "mfma_tile.h"
#include "mx_format.h"

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantisation

// A thread takes 8 neighbours of a row, four threads a block.  A workgroup's 256
// threads take consecutive pieces of the matrix.
template <typename T>
__device__ __forceinline__ void load8_f32(const T* p, float* v) {
  if constexpr (sizeof(T) == 2) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    mt::load8(p, v);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* __restrict__ x, long long pieces, int per_row,
                                                          int K, int ld, uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scales) {
  const long long first = (long long)blockIdx.x * 256;
  const long long row0 = first / per_row;  // the same in every thread
  const int at = (int)(first - row0 * per_row) + threadIdx.x;
  const long long row = row0 + at / per_row;
  const int c = at % per_row;
  const bool in = first + threadIdx.x < pieces;  // a block's four threads alike
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (in) load8_f32(x + row * K + c * 8, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mx::abs_bits(v[i]));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lane ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lane ^ 2
  if (!in) return;
  const uint32_t byte = mx::scale_of(m);
  const float inv = mx::inverse(byte);
  uint32_t w = mx::codes4<false>(0u, v[0], v[1], v[2], v[3], inv);
  w = mx::codes4<true>(w, v[4], v[5], v[6], v[7], inv);
  *reinterpret_cast<uint32_t*>(q + row * (K / 2) + c * 4) = byte == 255u ? 0u : w;
  uint8_t* s = scales + row * ld;
  if ((c & 3) == 0) s[c >> 2] = (uint8_t)byte;
  for (int i = K / mx::BLOCK + c; i < ld; i += per_row) s[i] = 0;
}

template <typename T>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ q,
                                                            const uint8_t* __restrict__ scales, long long pieces,
                                                            int per_row, int K, int ld, T* __restrict__ x) {
  const long long first = (long long)blockIdx.x * 256;
  const long long row0 = first / per_row;
  const int at = (int)(first - row0 * per_row) + threadIdx.x;
  const long long row = row0 + at / per_row;
  const int c = at % per_row;
  if (first + threadIdx.x >= pieces) return;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(q + row * (K / 2) + c * 4);
  const float f = mx::power(scales[row * ld + (c >> 2)]);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = (w >> (4 * i)) & 15u, e = (u >> 1) & 3u, m = u & 1u;
    const float a = e ? (float)((2 + m) << (e - 1)) * 0.5f : 0.5f * (float)m;
    v[i] = (u & 8u ? -a : a) * f;
  }
  mt::store8(x + row * K + c * 8, v);
}

// ---------------------------------------------------------------- grouped FFN

struct MxArgs {
  FfnSched s;
  const uint8_t* a;   // rows' codes [.][K/2]
  const uint8_t* as;  // and scales [.][lda]
  const uint8_t* w;   // [E][N][K/2]
  const uint8_t* ws;  // [E][N][lda]
  uint8_t* q;         // gate/up: activations' codes [rows][inter/2]
  uint8_t* qs;        // and scales [rows][ldq]
  void* y;            // down: [rows][N]
  int rows, K, N, lda, inter, ldq, ntn;
};

__device__ __forceinline__ f32x16_t mx_mfma(uint4 a, uint4 b, f32x16_t c, int sa, int sb) {
  const i32x8_t x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

// Block of 32 activations of a row, 16 in this lane (columns 8 i + 4 fh + j) and
// 16 in the lane 32 away: the row's scale byte, and codes 16 fh .. 16 fh + 15.
__device__ __forceinline__ uint2 act_block(const f32x16_t& g, const f32x16_t& u, uint32_t& byte) {
  float a[16];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = silu_f32(g[i]) * u[i];
    m = max(m, mx::abs_bits(a[i]));
  }
  const auto mm = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  byte = mx::scale_of(max(mm[0], mm[1]));
  const float inv = mx::inverse(byte);
  uint32_t lo = mx::codes4<false>(0u, a[0], a[1], a[2], a[3], inv);
  lo = mx::codes4<true>(lo, a[4], a[5], a[6], a[7], inv);
  uint32_t hi = mx::codes4<false>(0u, a[8], a[9], a[10], a[11], inv);
  hi = mx::codes4<true>(hi, a[12], a[13], a[14], a[15], inv);
  if (byte == 255u) lo = hi = 0u;
  // the lane halves trade: columns 0..15 to the lower, 16..31 to the upper
  const auto r = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
  return make_uint2((r[0] & 0xffffu) | (r[1] << 16), (r[0] >> 16) | (r[1] & 0xffff0000u));
}

// A row's 32 columns to memory: 16 in this lane, 16 in the lane 32 away.
__device__ __forceinline__ void store_block(uint16_t* o, const f32x16_t& a, int fh) {
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    uint32_t x0 = bf16x2_pack(a[q * 4], a[q * 4 + 1]), x1 = bf16x2_pack(a[q * 4 + 2], a[q * 4 + 3]);
    uint32_t y0 = bf16x2_pack(a[q * 4 + 4], a[q * 4 + 5]), y1 = bf16x2_pack(a[q * 4 + 6], a[q * 4 + 7]);
    const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
    *reinterpret_cast<uint4*>(o + q * 8 + fh * 8) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
  }
}
__device__ __forceinline__ void store_block(float* o, const f32x16_t& a, int fh) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<float4*>(o + q * 8 + fh * 4) = make_float4(a[q * 4], a[q * 4 + 1], a[q * 4 + 2], a[q * 4 + 3]);
}

// Tile of 64 rows x 64 columns, four waves.  DOWN: rows are the activations',
// columns y's; else rows through the map, columns the gate's and the up's.
template <bool DOWN, typename T>
__global__ __launch_bounds__(256) void mx_tile_kernel(MxArgs p) {
  const int n = *p.s.n_mtiles, t = blockIdx.x;
  if (t >= n * p.ntn) return;
  const int mt_ = t / p.ntn, nt = t % p.ntn;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 31, fh = lane >> 5;
  const int e = p.s.mt_e[mt_], v0 = p.s.mt_v0[mt_] + (wave >> 1) * 32, end = p.s.eoff[e + 1];
  const int c0 = nt * 64 + (wave & 1) * 32;  // the wave's columns
  const int cols = DOWN ? p.N : p.inter;
  if (v0 >= end || c0 >= cols) return;
  const int v = v0 + fr < end ? v0 + fr : v0;
  const size_t ar = DOWN ? v : p.s.asrc[v], br = (size_t)e * p.N + c0 + fr;
  const uint8_t* a = p.a + ar * (p.K / 2);
  const uint8_t* as = p.as + ar * p.lda;
  const uint8_t* b = p.w + br * (p.K / 2);
  const uint8_t* bs = p.ws + br * p.lda;
  const size_t up = (size_t)p.inter * (p.K / 2), ups = (size_t)p.inter * p.lda;
  f32x16_t acc, acc2;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = acc2[i] = 0.f;
  for (int k0 = 0; k0 < p.K; k0 += 64) {
    const int k = k0 + fh * 32;
    const bool in = k < p.K;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 fa = in ? *reinterpret_cast<const uint4*>(a + k / 2) : zero;
    const uint4 fb = in ? *reinterpret_cast<const uint4*>(b + k / 2) : zero;
    const int sa = in ? as[k / 32] : 0, sb = in ? bs[k / 32] : 0;
    acc = mx_mfma(fb, fa, acc, sb, sa);
    if constexpr (!DOWN) {
      const uint4 fu = in ? *reinterpret_cast<const uint4*>(b + up + k / 2) : zero;
      acc2 = mx_mfma(fu, fa, acc2, in ? bs[ups + k / 32] : 0, sa);
    }
  }
  if constexpr (DOWN) {
    if (v0 + fr < end) store_block(static_cast<T*>(p.y) + (size_t)p.s.rowmap[v] * p.N + c0, acc, fh);
  } else {
    uint32_t byte;
    const uint2 o = act_block(acc, acc2, byte);
    if (v0 + fr < end) {
      *reinterpret_cast<uint2*>(p.q + (size_t)v * (p.inter / 2) + c0 / 2 + fh * 8) = o;
      if (fh == 0) p.qs[(size_t)v * p.ldq + c0 / 32] = (uint8_t)byte;
    }
  }
}

// ---------------------------------------------------------------- host

struct MxLayout {
  size_t xq, xs, aq, as, total;
};
MxLayout mx_layout(int rows_x, int rows, int num_groups, int E, int d, int inter) {
  MxLayout l;
  l.xq = sched_layout(rows, num_groups, E, 0, MOELB_BF16, nullptr, nullptr);
  l.xs = l.xq + moelb_align256((size_t)rows_x * (d / 2));
  l.aq = l.xs + moelb_align256((size_t)rows_x * mx::scale_bytes(d));
  l.as = l.aq + moelb_align256((size_t)rows * (inter / 2));
  l.total = l.as + moelb_align256((size_t)rows * mx::scale_bytes(inter));
  return l;
}

constexpr int MAX_WIDTH = 1 << 19;

bool sizes_ok(int rows_x, int rows, int num_groups, int E, int d, int inter) {
  return rows >= 0 && rows_x >= 0 && num_groups >= 1 && num_groups <= 32768 && E >= 1 && E <= MOELB_MAX_E && d >= 32 &&
         d % 32 == 0 && d <= MAX_WIDTH && inter >= 32 && inter % 32 == 0 && inter <= MAX_WIDTH &&
         (size_t)rows_x * (d / 2) < mt::MAX_BYTES && (size_t)rows * (inter / 2) < mt::MAX_BYTES &&
         (size_t)inter * d < mt::MAX_BYTES && (size_t)rows * d * 4 < mt::MAX_BYTES;
}

bool aligned16(std::initializer_list<const void*> ps) {
  uintptr_t u = 0;
  for (const void* p : ps) u |= reinterpret_cast<uintptr_t>(p);
  return (u & 15) == 0;
}

template <typename T>
int launch_quantize(const void* x, long long rows, int K, uint8_t* q, uint8_t* scales, hipStream_t s) {
  const long long pieces = rows * (K / 8), blocks = (pieces + 255) / 256;
  if (blocks > (long long)moelb_most_blocks(256)) return MOELB_EINVAL;
  if (blocks == 0) return MOELB_OK;
  hipLaunchKernelGGL((mx_quantize_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const T*>(x), pieces,
                     K / 8, K, mx::scale_bytes(K), q, scales);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

template <typename T>
int run_ffn(const MxArgs& base, const void* x, int rows_x, int d, int inter, const uint8_t* w13, const uint8_t* w13s,
            const uint8_t* w2, const uint8_t* w2s, uint8_t* xq, uint8_t* xs, hipStream_t s, size_t mtiles) {
  int st = launch_quantize<T>(x, rows_x, d, xq, xs, s);
  if (st != MOELB_OK) return st;
  MxArgs p = base;
  p.a = xq, p.as = xs, p.w = w13, p.ws = w13s;
  p.K = d, p.N = 2 * inter, p.lda = mx::scale_bytes(d), p.ntn = (inter + 63) / 64;
  hipLaunchKernelGGL((mx_tile_kernel<false, T>), dim3((unsigned)(mtiles * p.ntn)), dim3(256), 0, s, p);
  MOELB_CHECK_LAUNCH();
  p.a = p.q, p.as = p.qs, p.w = w2, p.ws = w2s;
  p.K = inter, p.N = d, p.lda = p.ldq, p.ntn = (d + 63) / 64;
  hipLaunchKernelGGL((mx_tile_kernel<true, T>), dim3((unsigned)(mtiles * p.ntn)), dim3(256), 0, s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

}  // namespace

extern "C" int moelb_mx_scale_bytes(int K) { return K >= 32 && K % 32 == 0 ? mx::scale_bytes(K) : 0; }

extern "C" int moelb_mx_quantize(const void* x, long long rows, int K, int dtype, uint8_t* q, uint8_t* scales,
                                 void* stream) {
  if (rows < 0 || K < 32 || K % 32 != 0 || !moelb_dtype_ok(dtype)) return MOELB_EINVAL;
  if (rows > (1ll << 50) / K) return MOELB_EINVAL;
  if (!aligned16({x, q, scales})) return MOELB_EINVAL;
  if (rows > 0 && (!x || !q || !scales)) return MOELB_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dtype == MOELB_BF16 ? launch_quantize<uint16_t>(x, rows, K, q, scales, s)
                             : launch_quantize<float>(x, rows, K, q, scales, s);
}

extern "C" int moelb_mx_dequantize(const uint8_t* q, const uint8_t* scales, long long rows, int K, int dtype, void* x,
                                   void* stream) {
  if (rows < 0 || K < 32 || K % 32 != 0 || !moelb_dtype_ok(dtype)) return MOELB_EINVAL;
  if (rows > (1ll << 50) / K) return MOELB_EINVAL;
  if (!aligned16({x, q, scales})) return MOELB_EINVAL;
  if (rows > 0 && (!x || !q || !scales)) return MOELB_EINVAL;
  const long long pieces = rows * (K / 8), blocks = (pieces + 255) / 256;
  if (blocks > (long long)moelb_most_blocks(256)) return MOELB_EINVAL;
  if (blocks == 0) return MOELB_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == MOELB_BF16)
    hipLaunchKernelGGL((mx_dequantize_kernel<uint16_t>), dim3((unsigned)blocks), dim3(256), 0, s, q, scales, pieces,
                       K / 8, K, mx::scale_bytes(K), static_cast<uint16_t*>(x));
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<float>), dim3((unsigned)blocks), dim3(256), 0, s, q, scales, pieces, K / 8,
                       K, mx::scale_bytes(K), static_cast<float*>(x));
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

extern "C" size_t moelb_mx_grouped_ffn_workspace_bytes(int rows_x, int rows, int num_groups, int E, int d, int inter) {
  if (!sizes_ok(rows_x, rows, num_groups, E, d, inter)) return 0;
  return mx_layout(rows_x, rows, num_groups, E, d, inter).total;
}

extern "C" int moelb_mx_grouped_ffn(const void* x, int rows_x, int rows, const int32_t* group_off, int num_groups,
                                    int E, int G, int rank, const int32_t* gather, int gather_k, int d, int inter,
                                    int dtype, const uint8_t* w13, const uint8_t* w13_scales, const uint8_t* w2,
                                    const uint8_t* w2_scales, void* ws, size_t ws_bytes, void* y, void* stream) {
  if (!sizes_ok(rows_x, rows, num_groups, E, d, inter) || !moelb_dtype_ok(dtype)) return MOELB_EINVAL;
  if (rank >= 0 && (G < 1 || rank >= G || num_groups % E != 0)) return MOELB_EINVAL;
  if (gather && gather_k < 1) return MOELB_EINVAL;
  if (!group_off || !w13 || !w13_scales || !w2 || !w2_scales) return MOELB_EINVAL;
  if (rows > 0 && (!x || !y || rows_x < 1)) return MOELB_EINVAL;
  if (!aligned16({x, w13, w13_scales, w2, w2_scales, y})) return MOELB_EINVAL;
  const size_t mtiles = max_mtiles(rows, E), ntn = (size_t)((d > inter ? d : inter) + 63) / 64;
  if (mtiles * ntn > moelb_most_blocks(256)) return MOELB_EINVAL;
  const MxLayout l = mx_layout(rows_x, rows, num_groups, E, d, inter);
  if (!ws || !aligned16({ws}) || ws_bytes < l.total) return MOELB_EWORKSPACE;
  if (rows == 0) return MOELB_OK;
  char* base = static_cast<char*>(ws);
  MxArgs p = {};
  sched_layout(rows, num_groups, E, 0, MOELB_BF16, &p.s, base);
  p.q = reinterpret_cast<uint8_t*>(base + l.aq);
  p.qs = reinterpret_cast<uint8_t*>(base + l.as);
  p.y = y;
  p.rows = rows, p.inter = inter, p.ldq = mx::scale_bytes(inter);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int st = launch_schedule(group_off, num_groups, E, G, rank, rows, SCHED_MIN_BM, gather, gather_k, rows_x, p.s, s);
  if (st != MOELB_OK) return st;
  uint8_t* xq = reinterpret_cast<uint8_t*>(base + l.xq);
  uint8_t* xs = reinterpret_cast<uint8_t*>(base + l.xs);
  return dtype == MOELB_BF16
             ? run_ffn<uint16_t>(p, x, rows_x, d, inter, w13, w13_scales, w2, w2_scales, xq, xs, s, mtiles)
             : run_ffn<float>(p, x, rows_x, d, inter, w13, w13_scales, w2, w2_scales, xq, xs, s, mtiles);
}
