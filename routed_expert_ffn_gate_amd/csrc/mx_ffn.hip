// Experts in microscaled 4-bit floating point: quantisation, reading back, and
// the grouped FFN on tokens, activations and weights in that format.
//
// Definition (include/moelb.h, moelb_mx_quantize and moelb_mx_grouped_ffn): the
// OCP MX format with e2m1 elements; the FFN is moelb_grouped_ffn's (FreeBalance,
// "FreeBalance: Pre-Routing Online MoE Load Balancing via Residual Workload
// Prediction", section 2.1) with both factors of every product in it.
//
// Three launches: the schedule with the tokens' quantisation, gate/up with SwiGLU and
// the activations' quantisation as its epilogue, and down.  The products run on
// v_mfma_scale_f32_32x32x64_f8f6f4 over tiles streamed into LDS.  The weights'
// fragment is the instruction's first operand, so a lane ends with 16 columns of one
// row: a block's magnitude, codes and scale are formed between two lanes, without LDS.
//
// Bound by the weights' stream where an expert has few rows (512 tokens of 8, 128
// experts, d = 2048, inter = 768: 322 MB of weights in 80 us, 4.2 TB/s), and where it
// has hundreds by several parts that do not hide each other (16384 tokens of 8, 64
// experts, inter = 1024: 670 us, 2.5 PFLOP/s; registers alone reach 6.4): left out of a
// copy, the matrix instructions save 27 % of a dense gate/up product, the memory's loads
// 22, the fragments' reads of LDS and the epilogue 7 each, at 2.0-2.2 GHz.
#include <cmath>

#include "ffn_sched.h"
#include "mfma_tile.h"
#include "mx_format.h"

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantisation

// A thread takes 16 neighbours of a row, two threads a block.  A workgroup's 256
// threads take consecutive pieces of the matrix.  Bound by HBM: 131072 x 2048 bf16
// quantised in 121 us, read back in 110 (0.68 GB each: 5.6 and 6.2 TB/s).
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
__device__ __forceinline__ void quantize_pieces(int block, const T* __restrict__ x, long long pieces, int per_row, int K,
                                                int ld, uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  const long long first = (long long)block * 256;
  const long long row0 = first / per_row;  // the same in every thread
  const int at = (int)(first - row0 * per_row) + threadIdx.x;
  const long long row = row0 + at / per_row;
  const int c = at % per_row;
  const bool in = first + threadIdx.x < pieces;  // a block's two threads alike
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  if (in) {
    load8_f32(x + row * K + c * 16, v);
    load8_f32(x + row * K + c * 16 + 8, v + 8);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, mx::abs_bits(v[i]));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // lane ^ 1
  if (!in) return;
  const uint32_t byte = mx::scale_of(m);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* u = v + 8 * h;
    w[h] = mx::codes4<false>(0u, u[0], u[1], u[2], u[3], byte);
    w[h] = mx::codes4<true>(w[h], u[4], u[5], u[6], u[7], byte);
    if (byte == 255u) w[h] = 0u;
  }
  *reinterpret_cast<uint2*>(q + row * (K / 2) + c * 8) = make_uint2(w[0], w[1]);
  uint8_t* s = scales + row * ld;
  if ((c & 1) == 0) s[c >> 1] = (uint8_t)byte;
  for (int i = K / mx::BLOCK + c; i < ld; i += per_row) s[i] = 0;
}

template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* __restrict__ x, long long pieces, int per_row, int K,
                                                          int ld, uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scales) {
  quantize_pieces(blockIdx.x, x, pieces, per_row, K, ld, q, scales);
}

// The FFN's schedule and its tokens' quantisation in one launch: the first `ns`
// workgroups the one (it takes longer), the rest the other.  Two launches cost the
// small calls 2 us more.
template <typename T>
__global__ __launch_bounds__(256) void mx_prepare_kernel(int ns, const int32_t* __restrict__ group_off, int num_groups,
                                                         int E, int G, int rank, int rows, int BM,
                                                         const int32_t* __restrict__ gather, int gather_k, int rows_x,
                                                         FfnSched s, const T* __restrict__ x, long long pieces,
                                                         int per_row, int K, int ld, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ scales) {
  if ((int)blockIdx.x < ns)
    sched_rowmap(blockIdx.x, group_off, num_groups, E, G, rank, rows, BM, gather, gather_k, rows_x, s);
  else
    quantize_pieces(blockIdx.x - ns, x, pieces, per_row, K, ld, q, scales);
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
  const uint2 w = *reinterpret_cast<const uint2*>(q + row * (K / 2) + c * 8);
  const float f = mx::power(scales[row * ld + (c >> 1)]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
    mx::values8(h ? w.y : w.x, f, v);
    mt::store8(x + row * K + c * 16 + 8 * h, v);
  }
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
  int rows_x, rows, K, N, lda, inter, ldq, ntn;
};

// a . b over 64 k, the scales in byte 0 (HIGH: 2) of sa and sb.
template <bool HIGH>
__device__ __forceinline__ f32x16_t mx_mfma(uint4 a, uint4 b, f32x16_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, HIGH ? 2 : 0, (int)sa, HIGH ? 2 : 0, (int)sb);
}
__device__ __forceinline__ f32x16_t mx_mfma_at(uint4 a, uint4 b, f32x16_t c, uint32_t sa, uint32_t sb, int high) {
  return high ? mx_mfma<true>(a, b, c, sa, sb) : mx_mfma<false>(a, b, c, sa, sb);
}

// Block of 32 activations of a row, 16 in this lane (columns 8 i + 4 fh + j) and
// 16 in the lane 32 away: the row's scale byte, and codes 16 fh .. 16 fh + 15.  The
// hardware SiLU whatever the tokens' type: its error, |g| 2^-24 of the activation, only
// matters next to a border between two codes, as the fp32 sums' order does.
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
  uint32_t lo = mx::codes4<false>(0u, a[0], a[1], a[2], a[3], byte);
  lo = mx::codes4<true>(lo, a[4], a[5], a[6], a[7], byte);
  uint32_t hi = mx::codes4<false>(0u, a[8], a[9], a[10], a[11], byte);
  hi = mx::codes4<true>(hi, a[12], a[13], a[14], a[15], byte);
  if (byte == 255u) lo = hi = 0u;
  // the lane halves trade: columns 0..15 to the lower, 16..31 to the upper
  const auto r = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
  return make_uint2((r[0] & 0xffffu) | (r[1] << 16), (r[0] >> 16) | (r[1] & 0xffff0000u));
}

// A row's 32 columns to memory: 16 in this lane, 16 in the lane 32 away.
__device__ __forceinline__ void store_block(float* o, const f32x16_t& a, int fh) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<float4*>(o + q * 8 + fh * 4) = make_float4(a[q * 4], a[q * 4 + 1], a[q * 4 + 2], a[q * 4 + 3]);
}

// ---- the tile
//
// BM rows x BN weight rows a workgroup, NW waves, WM of them along the rows.  K
// steps of 256 (128 bytes a row) stream memory -> LDS into a ring of STAGES; the
// scales come 16 bytes a row, two steps at a time, into a ring of two beside them.
// Gate/up: the first half of the tile's weight rows are gate rows, the second the
// matching up rows, and a wave takes the same columns of both.  Loads go through
// buffer descriptors: a lane that asks for OUTSIDE gets zeros, which is how K ends
// inside a step (a zero code times any scale but NaN is 0).
//
// A step is four sub-steps of 64 k.  The barrier stands behind the last sub-step's
// reads: by then every wave has read the step's stage, which the refill takes, and
// has its part of the next step landed.
template <int BM_, int BN_, int NW_, int WM_, int STAGES_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, NW = NW_, WM = WM_, STAGES = STAGES_;
  static constexpr int THREADS = NW * 64, EU = BM * BN / NW > 4096 ? 1 : 2;
  static constexpr int WN = NW / WM, MI = BM / 32 / WM, NI = BN / 32 / WN;
  static constexpr int JA = BM / 8 / NW, JB = BN / 8 / NW;       // 1 KiB DMA instructions a wave and step
  static constexpr int J = JA + JB;
  static constexpr int JS = (BM + BN + 64 * NW - 1) / (64 * NW); // of scales, a wave and two steps
  static constexpr int STAGE = (BM + BN) * 128, CHUNK = JS * NW * 1024;
  static constexpr size_t LDS = (size_t)STAGES * STAGE + 2 * CHUNK;
};

// Virtual rows, expert and columns of a tile.
struct Place {
  int e, v0, end, nt;
};
__device__ __forceinline__ bool find_tile(const MxArgs& p, int bid, Place& o) {
  const int n = *p.s.n_mtiles, t = xcd_tile(bid, n * p.ntn);
  if (t < 0) return false;
  int mt_;
  grouped_tile(t, n, p.ntn, mt_, o.nt);
  o.e = p.s.mt_e[mt_];
  o.v0 = p.s.mt_v0[mt_];
  o.end = p.s.eoff[o.e + 1];
  return true;
}
// Memory row of the tile's row r: through the row map (gate/up), or the virtual row.
// Rows past the expert's end read some other row, and are not stored; the map's
// entries past the last row of all are not set, so what it gives is kept in range.
template <bool DOWN>
__device__ __forceinline__ uint32_t row_of(const MxArgs& p, const Place& o, int r) {
  const int v = min(o.v0 + r, p.rows - 1);
  return DOWN ? (uint32_t)v : min((uint32_t)p.s.asrc[v], (uint32_t)p.rows_x - 1u);
}
// Weight row (of the expert's N) of the tile's weight row r; past the last: row 0.
template <bool DOWN, int BN>
__device__ __forceinline__ uint32_t weight_of(const MxArgs& p, const Place& o, int r) {
  if (DOWN) {
    const int c = o.nt * BN + r;
    return (uint32_t)(c < p.N ? c : 0);
  }
  const int c = o.nt * (BN / 2) + r % (BN / 2), cc = c < p.inter ? c : 0;
  return (uint32_t)(r < BN / 2 ? cc : p.inter + cc);
}
// The tile's weight row where block ni of wave column wn starts.
template <bool DOWN, int BN, int NI>
__device__ __forceinline__ int block_row(int wn, int ni) {
  return DOWN ? (wn * NI + ni) * 32 : (wn * (NI / 2) + ni % (NI / 2)) * 32 + ni / (NI / 2) * (BN / 2);
}

// What a wave has in its accumulators to memory: block (mi, ni) is transposed,
// lane -> row lane % 32, element j -> column (j / 4) * 8 + (lane / 32) * 4 + j % 4.
// row0: the wave's first row of the tile.
// spare: LDS of the wave alone, through which bf16 rows leave in whole 128-byte
// lines (32-byte pieces straight from the accumulators: 308 against 285 us for the
// down product of 131072 rows, d = 2048, inter = 1024).
template <bool DOWN, typename T, int BN, int MI, int NI>
__device__ __forceinline__ void put_tile(const MxArgs& p, const Place& o, int row0, int wn,
                                         const f32x16_t (&acc)[MI][NI], char* spare) {
  const int lane = threadIdx.x & 63, fr = lane & 31, fh = lane >> 5;
  if constexpr (DOWN && sizeof(T) == 2) {
    static_assert(NI == 2, "a wave's 64 columns are a line");
    const int c0 = o.nt * BN + wn * 64, chunk = lane & 7;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      int to[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = o.v0 + row0 + mi * 32 + i * 8 + (lane >> 3);
        to[i] = v < o.end ? p.s.rowmap[v] : -1;
      }
      // row r of the block, 16-byte chunk c at c ^ (r % 8)
#pragma unroll
      for (int ni = 0; ni < 2; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16_t& a = acc[mi][ni];
          *reinterpret_cast<uint2*>(spare + fr * 128 + (((ni * 4 + q) ^ (fr & 7)) * 16) + fh * 8) =
              make_uint2(bf16x2_pack(a[q * 4], a[q * 4 + 1]), bf16x2_pack(a[q * 4 + 2], a[q * 4 + 3]));
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 3);
        const uint4 x = *reinterpret_cast<const uint4*>(spare + r * 128 + ((chunk ^ (r & 7)) * 16));
        if (to[i] >= 0 && c0 + chunk * 8 < p.N)
          store_nt16(static_cast<uint16_t*>(p.y) + (size_t)to[i] * p.N + c0 + chunk * 8, x);
      }
    }
    return;
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int v = o.v0 + row0 + mi * 32 + fr;
    const bool in = v < o.end;
    if constexpr (DOWN) {
      float* y = static_cast<float*>(p.y) + (size_t)(in ? p.s.rowmap[v] : 0) * p.N;
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        const int c = o.nt * BN + block_row<true, BN, NI>(wn, ni);
        if (in && c < p.N) store_block(y + c, acc[mi][ni], fh);
      }
    } else {
#pragma unroll
      for (int ni = 0; ni < NI / 2; ++ni) {
        const int c = o.nt * (BN / 2) + block_row<false, BN, NI>(wn, ni);
        uint32_t byte;
        const uint2 codes = act_block(acc[mi][ni], acc[mi][ni + NI / 2], byte);
        if (in && c < p.inter) {
          *reinterpret_cast<uint2*>(p.q + (size_t)v * (p.inter / 2) + c / 2 + fh * 8) = codes;
          uint8_t* s = p.qs + (size_t)v * p.ldq + c / 32;
          if (fh == 0) *s = (uint8_t)byte;
          if (fh == 1 && c + 32 == p.inter)  // the row's scales end here: zeros to the next 16 bytes
            for (int i = 1; c / 32 + i < p.ldq; ++i) s[i] = 0;
        }
      }
    }
  }
}

// NT: the weights' loads are marked non-temporal.
template <bool DOWN, bool NT, typename T, class G>
__global__ __launch_bounds__(G::THREADS, G::EU) void mx_stream_kernel(MxArgs p) {
  constexpr int BM = G::BM, BN = G::BN, MI = G::MI, NI = G::NI, JA = G::JA, JB = G::JB, J = G::J, JS = G::JS;
  constexpr int STAGE = G::STAGE, S = G::STAGES;
  extern __shared__ __align__(16) char smem[];
  Place o;
  if (!find_tile(p, blockIdx.x, o)) return;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / G::WN, wn = wave % G::WN, fr = lane & 31, fh = lane >> 5;
  const int KT = (p.K + 255) / 256, half = p.K / 2;
  const uint32_t rows_a = DOWN ? (uint32_t)p.rows : (uint32_t)p.rows_x;
  const mt::i32x4_t da = mt::descriptor(p.a, rows_a * (uint32_t)half);
  const mt::i32x4_t db = mt::descriptor(p.w + (size_t)o.e * p.N * half, (uint32_t)p.N * (uint32_t)half);
  const mt::i32x4_t dsa = mt::descriptor(p.as, rows_a * (uint32_t)p.lda);
  const mt::i32x4_t dsb = mt::descriptor(p.ws + (size_t)o.e * p.N * p.lda, (uint32_t)p.N * (uint32_t)p.lda);

  // DMA: instruction j of a wave fills the 8 LDS rows (J wave + j) * 8 ..; lane l
  // row l / 8 of them, 16-byte slot l % 8
  uint32_t aoff[JA], boff[JB], soff[JS];
  const int whole = half / 128;  // steps below it lie in K with all their bytes
  uint32_t tail = 0;             // in step `whole`: which instructions' pieces lie in K
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    const int r = (wave * JA + j) * 8 + (lane >> 3), c = mt::slot_of(r, lane & 7) * 16;
    aoff[j] = row_of<DOWN>(p, o, r) * (uint32_t)half + c;
    tail |= (uint32_t)(whole * 128 + c < half) << j;
  }
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const int r = (wave * JB + j) * 8 + (lane >> 3), c = mt::slot_of(r, lane & 7) * 16;
    boff[j] = weight_of<DOWN, BN>(p, o, r) * (uint32_t)half + c;
    tail |= (uint32_t)(whole * 128 + c < half) << (JA + j);
  }
#pragma unroll
  for (int j = 0; j < JS; ++j) {
    const int r = (wave * JS + j) * 64 + lane;  // the tile's rows, then its weight rows
    soff[j] = r < BM        ? row_of<DOWN>(p, o, r) * (uint32_t)p.lda
              : r < BM + BN ? weight_of<DOWN, BN>(p, o, r - BM) * (uint32_t)p.lda
                            : mt::OUTSIDE;
  }
  // instruction j (0 .. J-1) of step t
  auto issue = [&](int t, int j) {
    const uint32_t st = lds0 + (uint32_t)(t % S * STAGE);
    const bool in = t < whole || (tail >> j & 1);
    if (j < JA)
      mt::copy16(in ? aoff[j < JA ? j : 0] : mt::OUTSIDE, da, (uint32_t)t * 128u,
                 st + (uint32_t)((wave * JA + j) * 1024));
    else if (NT)
      mt::copy16_nt(in ? boff[j < JA ? 0 : j - JA] : mt::OUTSIDE, db, (uint32_t)t * 128u,
                    st + (uint32_t)(BM * 128 + (wave * JB + j - JA) * 1024));
    else
      mt::copy16(in ? boff[j < JA ? 0 : j - JA] : mt::OUTSIDE, db, (uint32_t)t * 128u,
                 st + (uint32_t)(BM * 128 + (wave * JB + j - JA) * 1024));
  };
  constexpr uint32_t SC = (uint32_t)(S * STAGE);
  auto issue_scales = [&](int c) {
#pragma unroll
    for (int j = 0; j < JS; ++j)  // an instruction's 64 rows are all of one operand: BM is a multiple of 64
      mt::copy16(soff[j], (wave * JS + j) * 64 < BM ? dsa : dsb, (uint32_t)c * 16u,
                 lds0 + SC + (uint32_t)((c & 1) * G::CHUNK + (wave * JS + j) * 1024));
  };
  int arow[MI], brow[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) arow[i] = (wm * MI + i) * 32 + fr;
#pragma unroll
  for (int i = 0; i < NI; ++i) brow[i] = block_row<DOWN, BN, NI>(wn, i) + fr;
  int at[4];  // byte of a row in sub-step ks: rows are a multiple of 32 and fr
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) at[ks] = mt::slot_of(fr, ks * 2 + fh) * 16;
  f32x16_t acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0.f;
  issue_scales(0);
  if (KT > 2) issue_scales(1);
  for (int t = 0; t < S && t < KT; ++t)
#pragma unroll
    for (int j = 0; j < J; ++j) issue(t, j);
  mt::wait_stages<J, S - 1>(min(S, KT) - 1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  for (int t = 0; t < KT; ++t) {
    const char* st = smem + t % S * STAGE;
    const char* sc = smem + SC + ((t >> 1) & 1) * G::CHUNK + (t & 1) * 8;
    // scales: bytes 2 ks + fh of a row's eight are those of sub-step ks
    uint32_t sa[MI][2], sb[NI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const uint2 v = *reinterpret_cast<const uint2*>(sc + arow[i] * 16);
      sa[i][0] = v.x >> (8 * fh), sa[i][1] = v.y >> (8 * fh);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint2 v = *reinterpret_cast<const uint2*>(sc + (BM + brow[i]) * 16);
      sb[i][0] = v.x >> (8 * fh), sb[i][1] = v.y >> (8 * fh);
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint4 fa[MI], fb[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) fb[i] = *reinterpret_cast<const uint4*>(st + BM * 128 + brow[i] * 128 + at[ks]);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = *reinterpret_cast<const uint4*>(st + arow[i] * 128 + at[ks]);
      if (ks == 3 && t + 1 < KT) {
        // lgkmcnt(0): this wave's reads of step t are done before its stage is refilled
        mt::wait_stages<J, S - 2>(min(S - 2, KT - 2 - t));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if ((t & 1) && t + 3 < KT) issue_scales((t + 3) / 2);
      }
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = mx_mfma_at(fb[ni], fa[mi], acc[mi][ni], sb[ni][ks >> 1], sa[mi][ks >> 1], ks & 1);
        if (ks == 3 && t + S < KT) {
#pragma unroll
          for (int j = mi; j < J; j += MI) issue(t + S, j);
        }
      }
    }
  }
  // the stage of the last step but one: every wave is past it, and nothing refills it
  char* spare = smem + (KT + S - 2) % S * STAGE + wave * (STAGE / G::NW);
  put_tile<DOWN, T, BN, MI, NI>(p, o, wm * MI * 32, wn, acc, spare);
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
         (size_t)inter * d < mt::MAX_BYTES;
}

bool aligned16(std::initializer_list<const void*> ps) {
  uintptr_t u = 0;
  for (const void* p : ps) u |= reinterpret_cast<uintptr_t>(p);
  return (u & 15) == 0;
}

template <typename T>
int launch_quantize(const void* x, long long rows, int K, uint8_t* q, uint8_t* scales, hipStream_t s) {
  const long long pieces = rows * (K / 16), blocks = (pieces + 255) / 256;
  if (blocks > (long long)moelb_most_blocks(256)) return MOELB_EINVAL;
  if (blocks == 0) return MOELB_OK;
  hipLaunchKernelGGL((mx_quantize_kernel<T>), dim3((unsigned)blocks), dim3(256), 0, s, static_cast<const T*>(x), pieces,
                     K / 16, K, mx::scale_bytes(K), q, scales);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

// Tiles of 128 or 64 rows, both two workgroups a compute unit.  128 rows read the
// weights half as often where experts have the rows; 64 waste less of the matrix
// instructions and load three steps ahead where the weights' stream is the time.
// d = 2048, inter = 768, 128 experts (128 | 64): 32 rows an expert 100 | 89 us, 64
// rows 111 | 102, 128 rows 137 | 144; 64 experts, inter = 1024, 512 rows 190 | 235.
using Large = Tile<128, 128, 4, 2, 2>;
using Small = Tile<64, 128, 4, 2, 3>;
bool large_rows(int rows, int E) { return (size_t)rows >= (size_t)96 * E; }
// Where even the most row tiles leave half of the compute units without one, tiles of
// 64 weight rows: one token of 8 experts 17.9 -> 17.4 us, 16 tokens of one expert,
// 4096 x 4096, 26.0 -> 23.8.
using Narrow = Tile<64, 64, 2, 2, 4>;
bool narrow_columns(int rows, int E, int d, int inter) {
  const size_t mt = (size_t)rows / 64 + (rows < E ? rows : E);
  const size_t up = (size_t)(inter + 63) / 64, down = (size_t)(d + 127) / 128;
  return mt * (up > down ? up : down) <= 128;
}

template <bool DOWN, bool NT, typename T, class G>
int launch_tiles(MxArgs p, size_t mtiles, hipStream_t s) {
  if (!moelb_allow_lds(mx_stream_kernel<DOWN, NT, T, G>, G::LDS)) return MOELB_ELAUNCH;
  p.ntn = (p.N + G::BN - 1) / G::BN;
  if (!DOWN) p.ntn = (p.inter + G::BN / 2 - 1) / (G::BN / 2);
  hipLaunchKernelGGL((mx_stream_kernel<DOWN, NT, T, G>), dim3((unsigned)(mtiles * p.ntn + 8)), dim3(G::THREADS), G::LDS,
                     s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

// NT: gate and up weights marked non-temporal.
template <bool NT, typename T, class G>
int launch_ffn(const MxArgs& base, int d, int inter, const uint8_t* w13, const uint8_t* w13s, const uint8_t* w2,
               const uint8_t* w2s, const uint8_t* xq, const uint8_t* xs, hipStream_t s, size_t mtiles) {
  MxArgs p = base;
  p.a = xq, p.as = xs, p.w = w13, p.ws = w13s;
  p.K = d, p.N = 2 * inter, p.lda = mx::scale_bytes(d);
  const int st = launch_tiles<false, NT, T, G>(p, mtiles, s);
  if (st != MOELB_OK) return st;
  p.a = p.q, p.as = p.qs, p.w = w2, p.ws = w2s;
  p.K = inter, p.N = d, p.lda = p.ldq;
  return launch_tiles<true, false, T, G>(p, mtiles, s);
}

// 64-row tiles that stream more weights than the 256 MB memory-side cache holds read
// the gate's and the up's non-temporally: no later call finds them there, and the
// activations and W2 stay.  512 tokens over 128 experts (322 MB) 86 -> 80 us, 64 tokens
// 76 -> 72.  Weights that fit are left alone (64 experts, 213 MB, called again at once:
// 56 us, non-temporal 65; 16 tokens over about 81 of 128 experts: 46 and 50), and so is
// W2, which the tiles of an expert share (all weights non-temporal: 85 us).  Counted are
// the experts that so many rows reach when each falls on any of them alike.
bool streams_weights(int rows, int E, int d, int inter) {
  const double experts = -E * std::expm1(-(double)rows / E);
  return experts * 3 * inter * d / 32 * 17 > 256.0 * (1 << 20);
}

struct Groups {
  const int32_t* off;
  int num, E, G, rank;
  const int32_t* gather;
  int gather_k;
};

template <typename T>
int run_ffn(const MxArgs& p, const Groups& g, const void* x, int d, int inter, const uint8_t* w13, const uint8_t* w13s,
            const uint8_t* w2, const uint8_t* w2s, uint8_t* xq, uint8_t* xs, hipStream_t s) {
  const bool large = large_rows(p.rows, g.E);
  const int bm = large ? Large::BM : Small::BM;
  const long long pieces = (long long)p.rows_x * (d / 16), nq = (pieces + 255) / 256;
  const int ns = (p.rows + 255) / 256;
  if (g.num <= SCHED_FUSED_GROUPS && ns + nq <= (long long)moelb_most_blocks(256)) {
    hipLaunchKernelGGL((mx_prepare_kernel<T>), dim3((unsigned)(ns + nq)), dim3(256), 0, s, ns, g.off, g.num, g.E,
                       g.G < 1 ? 1 : g.G, g.rank, p.rows, bm, g.gather, g.gather_k, p.rows_x, p.s,
                       static_cast<const T*>(x), pieces, d / 16, d, mx::scale_bytes(d), xq, xs);
    MOELB_CHECK_LAUNCH();
  } else {
    int st = launch_schedule(g.off, g.num, g.E, g.G, g.rank, p.rows, bm, g.gather, g.gather_k, p.rows_x, p.s, s);
    if (st != MOELB_OK) return st;
    st = launch_quantize<T>(x, p.rows_x, d, xq, xs, s);
    if (st != MOELB_OK) return st;
  }
  const size_t mtiles = (size_t)(p.rows + bm - 1) / bm + g.E;
  if (large) return launch_ffn<false, T, Large>(p, d, inter, w13, w13s, w2, w2s, xq, xs, s, mtiles);
  if (narrow_columns(p.rows, g.E, d, inter))
    return launch_ffn<false, T, Narrow>(p, d, inter, w13, w13s, w2, w2s, xq, xs, s, mtiles);
  return streams_weights(p.rows, g.E, d, inter)
             ? launch_ffn<true, T, Small>(p, d, inter, w13, w13s, w2, w2s, xq, xs, s, mtiles)
             : launch_ffn<false, T, Small>(p, d, inter, w13, w13s, w2, w2s, xq, xs, s, mtiles);
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
  const long long pieces = rows * (K / 16), blocks = (pieces + 255) / 256;
  if (blocks > (long long)moelb_most_blocks(256)) return MOELB_EINVAL;
  if (blocks == 0) return MOELB_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == MOELB_BF16)
    hipLaunchKernelGGL((mx_dequantize_kernel<uint16_t>), dim3((unsigned)blocks), dim3(256), 0, s, q, scales, pieces,
                       K / 16, K, mx::scale_bytes(K), static_cast<uint16_t*>(x));
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<float>), dim3((unsigned)blocks), dim3(256), 0, s, q, scales, pieces, K / 16,
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
  const size_t mtiles = max_mtiles(rows, E), ntn = (size_t)((d > inter ? d : inter) + 63) / 64 + 1;
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
  p.rows_x = rows_x, p.rows = rows, p.inter = inter, p.ldq = mx::scale_bytes(inter);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Groups g = {group_off, num_groups, E, G, rank, gather, gather_k};
  uint8_t* xq = reinterpret_cast<uint8_t*>(base + l.xq);
  uint8_t* xs = reinterpret_cast<uint8_t*>(base + l.xs);
  return dtype == MOELB_BF16 ? run_ffn<uint16_t>(p, g, x, d, inter, w13, w13_scales, w2, w2_scales, xq, xs, s)
                             : run_ffn<float>(p, g, x, d, inter, w13, w13_scales, w2, w2_scales, xq, xs, s);
}
