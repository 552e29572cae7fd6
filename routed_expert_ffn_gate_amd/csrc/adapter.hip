// A shared projection with the low-rank adapters of many requests beside it.
//
//   y[t] = x[t] W^T + scale_a (x[t] A_a^T) B_a^T,  a = ids[t]
// (no second term for a token without an adapter), optionally gated: W and B_a
// hold gate rows and then up rows, y = silu(gate) * up.  It stands where the
// layer's always-on shared expert stands, whose projections every request
// shares while its adapter is the request's own.
//
// The low products low[t] = scale_a x[t] A_a^T (r values a token) are formed
// first, then y:
//  * Prompts (adapter_tile_kernel): the product x W^T on the tile of
//    mfma_tile.h.  Where all tokens of a tile have one adapter, low and B_a are
//    further K steps of it (one, up to rank 64).  Elsewhere low B_a^T is added to
//    the accumulators afterwards for every adapter that occurs among a wave's
//    rows, fragments straight from memory.  An accumulator lane belongs to one
//    token, so a lane whose token has another adapter keeps its value: nothing
//    of one request's adapter, NaN or infinity included, reaches another's
//    tokens (as a shared K step with zeros for the other tokens would let it).
//    Its low products come from a launch of their own, in the storage type (an
//    operand of the second product, off by half a step of the adapter's small
//    share of y; few tokens keep them in fp32, so a token's last bit can follow
//    from the size of its batch).
//  * Few tokens (up to 256): the bytes of W and of the adapters in use bound it,
//    so the work is cut for many loads in flight: 64 rows of W x a part of k a
//    workgroup, v_mfma_f32_16x16x32_bf16 straight from registers, with the low
//    products' workgroups in the same launch; fp32 partial sums and low products
//    go through the workspace to a second launch, which adds them in order and
//    forms the rank-r products.
//  * One to four tokens with few ranks: one launch.  Every workgroup takes 16
//    rows of W and forms the low products itself (A_a of a token is as small as
//    its rows of W, and comes from L2).
// fp32 has the same forms on the fp32 tile: one to four tokens in one launch,
// few tokens with the adapters in the sum's kernel, else a walk over the tile's
// adapters; k is cut into parts wherever a call has fewer tiles than the card
// has compute units.
//
// Measured, bf16: one token, 2048 x 2048, r = 16: 5.8 us; 64 requests with an
// adapter each, 4096 x 4096 gated, r = 16: 11.3 us (4.4 TB/s of W and adapters)
// and 4.2 us for the second launch; 8192 tokens of 16 requests, 4096 x 4096, r =
// 64: low products 22 + 6 us, y 253 us (matrix units busy 0.59; 217 us is a
// library product of W alone).  Tokens in no order cost a walk over a tile's
// adapters: 512 tokens of 8 requests, r = 64, 50 us, each with an adapter of its
// own 359; 8192 tokens over 16 adapters at random 959 us, over 64 (r = 16) 1521.
// Few tokens of large ranks are bound by the second launch's reads of B: 64
// tokens, gated, r = 16, 64, 256: 16, 25, 70 us; 256 tokens: r = 16 34, r = 256 219.
#include "mfma_tile.h"

namespace {

struct AdapterArgs {
  const void* x;
  const void* w;
  const int32_t* ids;
  const void* a;
  const void* b;
  const float* scale;
  void* low;    // [T][r]; fp32 for few tokens, else the storage type
  float* part;  // few tokens: [splits][T][d_out]; prompts: [splits][T][r]
  void* y;
  int Ttok, d_in, d_out, n, r, ntn, splits, nbase;
  int first;  // number of this launch's first workgroup (launch_blocks)
};
__device__ __forceinline__ unsigned block_of(const AdapterArgs& p) { return (unsigned)p.first + blockIdx.x; }

__device__ __forceinline__ uint32_t bytes32(size_t n) { return n < mt::MAX_BYTES ? (uint32_t)n : (uint32_t)mt::MAX_BYTES; }
__device__ __forceinline__ int id_of(const AdapterArgs& p, int t) {
  const int id = p.n > 0 ? p.ids[t] : -1;
  return id >= 0 && id < p.n ? id : -1;
}

__device__ __forceinline__ void load_vec(const uint16_t* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_vec(const float* p, float (&v)[8]) { mt::load8(p, v); }

// Eight values at k of a lane's row (its own k offset kc is in the pointer), or
// zeros from k1 on; the address stays inside the row either way.
__device__ __forceinline__ bf16x8_t frag_at(const uint16_t* row, int k, int kc, int k1) {
  const bool in = k + kc < k1;
  const uint4 v = *reinterpret_cast<const uint4*>(row + (in ? k : -kc));
  return __builtin_bit_cast(bf16x8_t, in ? v : make_uint4(0, 0, 0, 0));
}

// ---------------------------------------------------------------- low = scale x A^T

// low in fp32: a wave per token and R ranks, dot products over d_in, 8 values a
// lane and step.
template <typename T, int WAVES, int R>
__device__ __forceinline__ void low_rows(const AdapterArgs& p, int block) {
  const long long wv = (long long)block * WAVES + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, per = p.r / R;
  const int t = (int)(wv / per), rr = (int)(wv % per) * R;
  if (t >= p.Ttok) return;
  const int id = id_of(p, t);
  if (id < 0) return;
  const T* x = static_cast<const T*>(p.x) + (size_t)t * p.d_in;
  const T* a = static_cast<const T*>(p.a) + ((size_t)id * p.r + rr) * p.d_in;
  float s[R][2];
#pragma unroll
  for (int j = 0; j < R; ++j) s[j][0] = s[j][1] = 0.f;
#pragma unroll 8 / R
  for (int k = lane * 8; k < p.d_in; k += MOELB_WAVE * 8) {
    float u[8], w[R][8];
    load_vec(x + k, u);
#pragma unroll
    for (int j = 0; j < R; ++j) load_vec(a + (size_t)j * p.d_in + k, w[j]);
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i & 1] = fmaf(u[i], w[j][i], s[j][i & 1]);
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float v = s[j][0] + s[j][1];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, MOELB_WAVE);
    if (lane == 0) static_cast<float*>(p.low)[(size_t)t * p.r + rr + j] = v * p.scale[id];
  }
}

// fp32 prompts.
template <int R>
__global__ __launch_bounds__(256) void adapter_low_rows_f32_kernel(AdapterArgs p) {
  low_rows<float, 4, R>(p, (int)block_of(p));
}

// The adapter of all tokens t0 .. t0 + rows - 1 (up to T), -1 if they differ or
// have none.  Wave-uniform.
__device__ __forceinline__ int same_id(const AdapterArgs& p, int t0, int rows) {
  if (p.n <= 0) return -1;
  const int id = __builtin_amdgcn_readfirstlane(id_of(p, t0));
  bool other = id < 0;
  for (int i = threadIdx.x & 63; i < rows; i += MOELB_WAVE)
    if (t0 + i < p.Ttok && id_of(p, t0 + i) != id) other = true;
  return __ballot(other) ? -1 : id;
}

// Prompts: a workgroup takes 128 tokens (32 a wave), 64 ranks (blockIdx.z) and
// one part of k (blockIdx.y); its waves read the same rows of A_a together.
// Tokens of one adapter: the tile of mfma_tile.h (half its columns unused up to
// rank 64; fragments straight from memory, a row a lane, are served 16 bytes a
// cycle: 30 us against 21 at 8192 tokens, d_in = 4096, r = 64).  Others: a wave
// walks the adapters among its tokens, in token order, with such fragments, and
// keeps of each product the rows of that adapter's tokens.  Partial sums go to
// part[split][T][r].
constexpr int LOW_TOK = 128;

__global__ __launch_bounds__(256) void adapter_low_tile_kernel(AdapterArgs p) {
  extern __shared__ __align__(16) char smem[];
  const int steps64 = (p.d_in + 63) / 64, per64 = (steps64 + p.splits - 1) / p.splits;
  const int k0 = min(p.d_in, (int)blockIdx.y * per64 * 64), k1 = min(p.d_in, k0 + per64 * 64);
  const int same = same_id(p, blockIdx.x * LOW_TOK, LOW_TOK);
  if (same >= 0) {
    const int t0 = blockIdx.x * LOW_TOK, n0 = blockIdx.z * 64;
    mt::RowOp<2> oa, ob;
    oa.init(static_cast<const uint16_t*>(p.x) + k0, bytes32(((size_t)p.Ttok * p.d_in - k0) * 2), p.d_in, k1 - k0,
            [&](int i) { return min(t0 + i, p.Ttok - 1); });
    ob.init(static_cast<const uint16_t*>(p.a) + (size_t)same * p.r * p.d_in + k0,
            bytes32(((size_t)p.r * p.d_in - k0) * 2), p.d_in, k1 - k0,
            [&](int i) { return min(n0 + (i & 63), p.r - 1); });
    f32x16_t acc[2][2];
    mt::k_loop<2, false>(reinterpret_cast<uint16_t*>(smem), oa, ob, max(1, (k1 - k0 + 63) / 64), acc);
    mt::drain<2, false>(reinterpret_cast<uint16_t*>(smem), acc, [&](int i, int c, const float* v) {
      if (t0 + i < p.Ttok && c < 64 && n0 + c < p.r)
        mt::store8(p.part + ((size_t)blockIdx.y * p.Ttok + t0 + i) * p.r + n0 + c, v);
    });
    return;
  }
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * LOW_TOK + (threadIdx.x >> 6) * 32 + (lane & 31), r0 = blockIdx.z * 64;
  const int mine = t < p.Ttok ? id_of(p, t) : -1;
  const int kc = (lane >> 5) * 8;
  const uint16_t* xr = static_cast<const uint16_t*>(p.x) + (size_t)min(t, p.Ttok - 1) * p.d_in + kc;
  const bool two = p.r - r0 > 32;
  uint64_t left = __ballot(mine >= 0);
  while (left) {
    const int id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    left &= ~__ballot(mine == id);
    const uint16_t* a = static_cast<const uint16_t*>(p.a) + (size_t)id * p.r * p.d_in + kc;
    const uint16_t* a0 = a + (size_t)min(r0 + (lane & 31), p.r - 1) * p.d_in;
    const uint16_t* a1 = a + (size_t)min(r0 + 32 + (lane & 31), p.r - 1) * p.d_in;
    f32x16_t acc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[j][q] = 0.f;
    for (int k = k0; k < k1; k += 64) {  // four steps' loads in flight
      bf16x8_t fx[4], f0[4], f1[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        fx[u] = frag_at(xr, k + u * 16, kc, k1);
        f0[u] = frag_at(a0, k + u * 16, kc, k1);
        if (two) f1[u] = frag_at(a1, k + u * 16, kc, k1);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f0[u], fx[u], acc[0], 0, 0, 0);
        if (two) acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f1[u], fx[u], acc[1], 0, 0, 0);
      }
    }
    // lane: token lane % 32; element j: rank (j / 4) * 8 + (lane / 32) * 4 + j % 4
    if (mine == id) {
      float* o = p.part + ((size_t)blockIdx.y * p.Ttok + t) * p.r;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rr = r0 + j * 32 + q * 8 + (lane >> 5) * 4;
          const f32x4_t v = {acc[j][q * 4], acc[j][q * 4 + 1], acc[j][q * 4 + 2], acc[j][q * 4 + 3]};
          if (rr < p.r) *reinterpret_cast<f32x4_t*>(o + rr) = v;
        }
    }
  }
}

// low = scale x the parts' sum, in order; four values a thread.
__global__ __launch_bounds__(256) void adapter_low_sum_kernel(AdapterArgs p) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i / (p.r / 4)), c = (int)(i % (p.r / 4)) * 4;
  if (t >= p.Ttok) return;
  const int id = id_of(p, t);
  if (id < 0) return;
  const float* o = p.part + (size_t)t * p.r + c;
  const float sc = p.scale[id];
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) v += *reinterpret_cast<const f32x4_t*>(o + (size_t)s * p.Ttok * p.r);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.low) + (size_t)t * p.r + c) =
      make_uint2(bf16x2_pack(v[0] * sc, v[1] * sc), bf16x2_pack(v[2] * sc, v[3] * sc));
}

// ---------------------------------------------------------------- prompts

// A row operand that goes on, after its own K steps, with the r columns of a
// second matrix (low, or B_a).
template <int F>
struct LongRowOp {
  static constexpr bool COL = false;
  mt::RowOp<F> own, more;
  int first;
  __device__ __forceinline__ void begin(int) {}
  __device__ __forceinline__ void issue(int t, int j, uint32_t m0) const {
    if (t < first)
      own.issue(t, j, m0);
    else
      more.issue(t - first, j, m0);
  }
};

// acc += low B^T for the adapters among this wave's 32 F rows.  own[mi]: the
// adapter of row block mi's lane % 32-th token, -1: none.  brow(ni): row of B
// for this lane in column block ni.
template <int F, class Row>
__device__ __forceinline__ void add_adapters(const AdapterArgs& p, int split, const uint16_t* const (&low)[F],
                                             const int (&own)[F], Row brow, f32x16_t (&acc)[F][F]) {
  const int kc = ((threadIdx.x & 63) >> 5) * 8;
  int left[F];
#pragma unroll
  for (int mi = 0; mi < F; ++mi) left[mi] = own[mi];
  for (int i = 0;; ++i) {  // the i-th adapter is part i % splits'
    int id = -1;
#pragma unroll
    for (int mi = F - 1; mi >= 0; --mi) {
      const uint64_t some = __ballot(left[mi] >= 0);
      if (some) id = __builtin_amdgcn_readlane(left[mi], __builtin_ctzll(some));
    }
    if (id < 0) return;
    const uint16_t* b = static_cast<const uint16_t*>(p.b) + (size_t)id * p.d_out * p.r + kc;
    bool mine[F];
#pragma unroll
    for (int mi = 0; mi < F; ++mi) {
      mine[mi] = own[mi] == id;
      if (mine[mi]) left[mi] = -1;
    }
    if (i % p.splits != split) continue;
    for (int k = 0; k < p.r; k += 64) {
      bf16x8_t fa[F][4];
#pragma unroll
      for (int mi = 0; mi < F; ++mi)
#pragma unroll
        for (int u = 0; u < 4; ++u) fa[mi][u] = frag_at(low[mi], k + u * 16, kc, mine[mi] ? p.r : 0);
#pragma unroll
      for (int ni = 0; ni < F; ++ni) {
        const uint16_t* br = b + (size_t)brow(ni) * p.r;
        bf16x8_t fb[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) fb[u] = frag_at(br, k + u * 16, kc, p.r);
#pragma unroll
        for (int mi = 0; mi < F; ++mi) {
          f32x16_t v;
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = 0.f;
#pragma unroll
          for (int u = 0; u < 4; ++u) v = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[u], fa[mi][u], v, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < 16; ++q) v[q] = mine[mi] ? v[q] : 0.f;
          f32x16_t c = acc[mi][ni];
          asm volatile("" : "+v"(c));
#pragma unroll
          for (int q = 0; q < 16; ++q) c[q] += v[q];
          asm volatile("" : "+a"(c));
          acc[mi][ni] = c;
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_gated(T* y, const float* g, const float* u) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mt::silu_as<T>(g[i]) * u[i];
  mt::store8(y, v);
}

// Tile order: as the grouped FFN's, 8 token tiles x every column tile, dealt in
// contiguous ranges to the 8 XCDs.
__device__ __forceinline__ bool tile_of(const AdapterArgs& p, int B, int bid, int& mi, int& ni) {
  const int ntm = (p.Ttok + B - 1) / B, total = ntm * p.ntn;
  const int per = (total + 7) / 8;
  const int t = (bid & 7) * per + (bid >> 3);
  if (bid >> 3 >= per || t >= total) return false;
  const int group = t / (8 * p.ntn), gm = min(8, ntm - group * 8), local = t - group * 8 * p.ntn;
  ni = local / gm;
  mi = group * 8 + local % gm;
  return true;
}

// splits > 1: blockIdx.y takes a part of k, and of the adapters of a tile that
// has several; fp32 partial sums to part[split][T][d_out].
template <int F, bool GU>
__global__ __launch_bounds__(mt::THREADS) void adapter_tile_kernel(AdapterArgs p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  constexpr int B = 64 * F;
  int mi, ni;
  if (!tile_of(p, B, blockIdx.x, mi, ni)) return;
  const int split = blockIdx.y;
  const int steps = (p.d_in + mt::BK - 1) / mt::BK, ps = (steps + p.splits - 1) / p.splits;
  const int k0 = min(p.d_in, split * ps * mt::BK), k1 = min(p.d_in, k0 + ps * mt::BK);
  const int t0 = mi * B, n0 = ni * (GU ? B / 2 : B);
  const int out = GU ? p.d_out / 2 : p.d_out;
  auto trow = [&](int i) { return min(t0 + i, p.Ttok - 1); };
  auto wrow = [&](int i) {
    const int c = n0 + (GU ? i % (B / 2) : i);
    return (c < out ? c : 0) + (GU && i >= B / 2 ? out : 0);
  };
  // a tile of one adapter takes its ranks as further K steps (of the last part)
  const int id = same_id(p, t0, B);
  LongRowOp<F> oa, ob;
  oa.own.init(static_cast<const uint16_t*>(p.x) + k0, bytes32(((size_t)p.Ttok * p.d_in - k0) * 2), p.d_in, k1 - k0,
              trow);
  ob.own.init(static_cast<const uint16_t*>(p.w) + k0, bytes32(((size_t)p.d_out * p.d_in - k0) * 2), p.d_in, k1 - k0,
              wrow);
  oa.more.init(p.low, bytes32((size_t)p.Ttok * p.r * 2), p.r, p.r, trow);
  ob.more.init(static_cast<const uint16_t*>(p.b) + (size_t)max(id, 0) * p.d_out * p.r,
               bytes32((size_t)p.d_out * p.r * 2), p.r, p.r, wrow);
  oa.first = ob.first = max(1, (k1 - k0 + mt::BK - 1) / mt::BK);  // an empty part: a step of zeros
  f32x16_t acc[F][F];
  const bool more = id >= 0 && split == p.splits - 1;
  mt::k_loop<F, GU>(lds, oa, ob, oa.first + (more ? (p.r + mt::BK - 1) / mt::BK : 0), acc);
  if (p.n > 0 && id < 0) {
    const int lane = threadIdx.x & 63, wm = threadIdx.x >> 7, wn = (threadIdx.x >> 6) & 1;
    const uint16_t* low[F];
    int own[F];
#pragma unroll
    for (int mi = 0; mi < F; ++mi) {
      const int t = t0 + wm * 32 * F + mi * 32 + (lane & 31);
      own[mi] = t < p.Ttok ? id_of(p, t) : -1;
      low[mi] = static_cast<const uint16_t*>(p.low) + (size_t)min(t, p.Ttok - 1) * p.r + (lane >> 5) * 8;
    }
    add_adapters<F>(p, split, low, own, [&](int ni) { return wrow(mt::block_col<F, GU>(wn, ni) + (lane & 31)); }, acc);
  }
  uint16_t* y = static_cast<uint16_t*>(p.y);
  float* part = p.part + ((size_t)split * p.Ttok + t0) * p.d_out + n0;
  if constexpr (GU) {
    mt::drain<F, true>(lds, acc, [&](int r, int c, const float* g, const float* u) {
      if (t0 + r >= p.Ttok || n0 + c >= out) return;
      if (p.splits > 1) {
        mt::store8(part + (size_t)r * p.d_out + c, g);
        mt::store8(part + (size_t)r * p.d_out + out + c, u);
      } else {
        store_gated(y + (size_t)(t0 + r) * out + n0 + c, g, u);
      }
    });
  } else {
    mt::drain<F, false>(lds, acc, [&](int r, int c, const float* v) {
      if (t0 + r >= p.Ttok || n0 + c >= out) return;
      if (p.splits > 1)
        mt::store8(part + (size_t)r * p.d_out + c, v);
      else
        mt::store8(y + (size_t)(t0 + r) * out + n0 + c, v);
    });
  }
}

// fp32: the same sum on 64 x 64 tiles.  FEW (few tokens): blocks from nbase on
// form the low products and the adapters are left to the sum's kernel.  Parts of
// k as above.
template <bool GU, bool FEW>
__global__ __launch_bounds__(mt::S_THREADS) void adapter_tile_f32_kernel(AdapterArgs p) {
  __shared__ __align__(16) float lds[mt::STile<64>::FLOATS];
  __shared__ int tok[64];
  const unsigned bid = block_of(p);
  if (FEW && (int)bid >= p.nbase) {
    low_rows<float, mt::S_THREADS / MOELB_WAVE, 1>(p, bid - p.nbase);
    return;
  }
  const int tiles = p.nbase / p.splits, split = bid / tiles;  // tiles: a multiple of 8
  int mi, ni;
  if (!tile_of(p, 64, bid - split * tiles, mi, ni)) return;
  const int t0 = mi * 64, n0 = ni * (GU ? 32 : 64);
  const int out = GU ? p.d_out / 2 : p.d_out;
  const int per = ((p.d_in + 63) / 64 + p.splits - 1) / p.splits * 64;
  const int k0 = min(p.d_in, split * per), k1 = min(p.d_in, k0 + per);
  const float* x = static_cast<const float*>(p.x) + k0;
  const float* w = static_cast<const float*>(p.w) + k0;
  const float* low = static_cast<const float*>(p.low);
  auto wrow = [&](int i) {
    const int c = n0 + (GU ? i & 31 : i);
    return c < out ? c + (GU && i >= 32 ? out : 0) : -1;
  };
  f32x16_t acc;
  {
    auto pa = [&](int i, int k) { return t0 + i < p.Ttok ? x + (size_t)(t0 + i) * p.d_in + k : nullptr; };
    auto pb = [&](int i, int k) { return wrow(i) >= 0 ? w + (size_t)wrow(i) * p.d_in + k : nullptr; };
    mt::k_loop_f32<64, false, false>(lds, pa, pb, k1 - k0, acc);
  }
  if (!FEW && p.n > 0) {
    // every wave walks the tile's adapters (they load the rows together); a
    // lane whose token has another one keeps its value
    if (threadIdx.x < 64) tok[threadIdx.x] = t0 + (int)threadIdx.x < p.Ttok ? id_of(p, t0 + threadIdx.x) : -1;
    __syncthreads();
    int left = tok[threadIdx.x & 63];
    const int own = tok[(threadIdx.x >> 6 & 1) * 32 + (threadIdx.x & 31)];  // the lane's token
    int turn = 0;  // the parts take the adapters in turn
    for (uint64_t some = __ballot(left >= 0); some; some = __ballot(left >= 0)) {
      const int id = __builtin_amdgcn_readlane(left, __builtin_ctzll(some));
      if (left == id) left = -1;
      if (turn++ % p.splits != split) continue;
      const float* b = static_cast<const float*>(p.b) + (size_t)id * p.d_out * p.r;
      auto pa = [&](int i, int k) { return tok[i] == id ? low + (size_t)(t0 + i) * p.r + k : nullptr; };
      auto pb = [&](int i, int k) { return wrow(i) >= 0 ? b + (size_t)wrow(i) * p.r + k : nullptr; };
      f32x16_t more;
      __syncthreads();
      mt::k_loop_f32<64, false, false>(lds, pa, pb, p.r, more);
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[q] = own == id ? acc[q] + more[q] : acc[q];
    }
  }
  if (FEW || p.splits > 1) {
    float* part = p.part + (size_t)split * p.Ttok * p.d_out;
    mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) {
      if (t0 + r < p.Ttok && wrow(c) >= 0) mt::store8(part + (size_t)(t0 + r) * p.d_out + wrow(c), v);
    });
    return;
  }
  float* y = static_cast<float*>(p.y);
  if constexpr (GU) {
    mt::drain_f32<64, true>(lds, acc, [&](int r, int c, const float* g, const float* u) {
      if (t0 + r < p.Ttok && n0 + c < out) store_gated(y + (size_t)(t0 + r) * out + n0 + c, g, u);
    });
  } else {
    mt::drain_f32<64, false>(lds, acc, [&](int r, int c, const float* v) {
      if (t0 + r < p.Ttok && n0 + c < out) mt::store8(y + (size_t)(t0 + r) * out + n0 + c, v);
    });
  }
}

// ---------------------------------------------------------------- few tokens

// Base part: 64 rows of W x 16 NB tokens x one part of k.  W and
// x stream memory -> LDS in 64-wide K steps, three ahead (a row's 128 bytes by 8
// neighbouring lanes: read as fragments, a row a lane, they come at a quarter of
// the rate), the slots of a row XORed so that 16 rows' fragments lie on
// different banks; wave w takes rows 16 w .., all tokens.  Blocks from nbase on
// form the low products.
constexpr int FEW_STAGES = 4;

template <int NB>
__global__ __launch_bounds__(256) void adapter_few_kernel(AdapterArgs p) {
  const unsigned bid = block_of(p);
  if ((int)bid >= p.nbase) {
    low_rows<uint16_t, 4, 1>(p, bid - p.nbase);
    return;
  }
  constexpr int TOK = 16 * NB, STAGE = (64 + TOK) * 64;  // elements
  constexpr int NX = NB > 1 ? NB / 2 : 1;                // DMA instructions of x a wave and stage
  __shared__ __align__(16) uint16_t lds[FEW_STAGES * STAGE];
  const uint32_t lds_u32 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // a token block's workgroups of one W block are neighbours: they share its rows in L2
  const int tb = (p.Ttok + TOK - 1) / TOK;
  const int split = bid / tb % p.splits, n0 = bid / tb / p.splits * 64, t0 = bid % tb * TOK;
  const int steps = (p.d_in + 63) / 64, per = (steps + p.splits - 1) / p.splits;
  const int s0 = min(steps, split * per), n = min(steps, s0 + per) - s0;
  const mt::i32x4_t ws = mt::descriptor(p.w, bytes32((size_t)p.d_out * p.d_in * 2));
  const mt::i32x4_t xs = mt::descriptor(p.x, bytes32((size_t)p.Ttok * p.d_in * 2));
  // DMA block b (8 rows): lane -> row lane / 8, slot lane % 8 <- chunk slot ^ swizzle
  uint32_t woff[2], xoff[NX];
  int wck[2], xck[NX], xblk[NX];
  auto chunk = [&](int r) { return (lane & 7) ^ (((r >> 1) ^ (r << 2)) & 7); };
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = (wave * 2 + j) * 8 + (lane >> 3);
    wck[j] = chunk(r) * 8;
    woff[j] = ((uint32_t)min(n0 + r, p.d_out - 1) * (uint32_t)p.d_in + wck[j]) * 2u;
  }
#pragma unroll
  for (int j = 0; j < NX; ++j) {
    xblk[j] = NB > 1 ? wave * NX + j : wave & 1;  // NB = 1: waves 2, 3 write what 0, 1 write
    const int r = xblk[j] * 8 + (lane >> 3);
    xck[j] = chunk(r) * 8;
    xoff[j] = ((uint32_t)min(t0 + r, p.Ttok - 1) * (uint32_t)p.d_in + xck[j]) * 2u;
  }
  auto issue = [&](int i) {
    const uint32_t st = lds_u32 + (uint32_t)((i % FEW_STAGES) * STAGE) * 2u;
    const int k = (s0 + i) * 64;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      mt::copy16(wck[j] + k < p.d_in ? woff[j] : mt::OUTSIDE, ws, (uint32_t)k * 2u,
                 st + (uint32_t)((wave * 2 + j) * 512) * 2u);
#pragma unroll
    for (int j = 0; j < NX; ++j)
      mt::copy16(xck[j] + k < p.d_in ? xoff[j] : mt::OUTSIDE, xs, (uint32_t)k * 2u,
                 st + (uint32_t)(64 * 64 + xblk[j] * 512) * 2u);
  };
  f32x4_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < FEW_STAGES - 1 && i < n; ++i) issue(i);
  const int fr = lane & 15, fc = lane >> 4, sw = ((fr >> 1) ^ (fr << 2)) & 7;
  for (int i = 0; i < n; ++i) {
    // stage i landed (at most the two after it are in flight), and every wave
    // has read stage i - 1, whose place the next load takes
    constexpr int V = 2 + NX;
    if (i + 2 < n)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * V) : "memory");
    else if (i + 1 < n)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(V) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (i + FEW_STAGES - 1 < n) issue(i + FEW_STAGES - 1);
    const uint16_t* st = lds + (i % FEW_STAGES) * STAGE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = ((h * 4 + fc) ^ sw) * 8;
      const bf16x8_t fw = *reinterpret_cast<const bf16x8_t*>(st + (wave * 16 + fr) * 64 + c);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const bf16x8_t fx = *reinterpret_cast<const bf16x8_t*>(st + (64 + j * 16 + fr) * 64 + c);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw, fx, acc[j], 0, 0, 0);
      }
    }
  }
  // lane: token lane % 16 of block j, rows 16 wave + (lane / 16) * 4 ..
  const int c0 = n0 + wave * 16 + fc * 4;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int tok = t0 + j * 16 + fr;
    if (tok < p.Ttok && c0 < p.d_out)
      *reinterpret_cast<f32x4_t*>(p.part + ((size_t)split * p.Ttok + tok) * p.d_out + c0) = acc[j];
  }
}

// Two rows of W a thread (a gate and its up row, or two neighbours): their
// partial sums in order, and low . B rows.
template <typename T, bool GU>
__global__ __launch_bounds__(256) void adapter_few_sum_kernel(AdapterArgs p) {
  const int out = GU ? p.d_out / 2 : p.d_out, per = GU ? out : out / 2;
  const long long i = (long long)block_of(p) * 256 + threadIdx.x;
  const int t = (int)(i / per), c = (int)(i % per);
  if (t >= p.Ttok) return;
  const int c0 = GU ? c : 2 * c, c1 = GU ? out + c : 2 * c + 1;
  const int id = id_of(p, t);
  const float* part = p.part + (size_t)t * p.d_out;
  float v0 = 0.f, v1 = 0.f;
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float* q = part + (size_t)s * p.Ttok * p.d_out;
    v0 += q[c0];
    v1 += q[c1];
  }
  if (id >= 0) {
    const float* low = static_cast<const float*>(p.low) + (size_t)t * p.r;
    const T* b = static_cast<const T*>(p.b) + (size_t)id * p.d_out * p.r;
#pragma unroll 2
    for (int k = 0; k < p.r; k += 8) {
      float l[8], u[8], w[8];
      mt::load8(low + k, l);
      load_vec(b + (size_t)c0 * p.r + k, u);
      load_vec(b + (size_t)c1 * p.r + k, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v0 = fmaf(l[q], u[q], v0);
        v1 = fmaf(l[q], w[q], v1);
      }
    }
  }
  T* y = static_cast<T*>(p.y) + (size_t)t * out;
  if constexpr (GU)
    Elem<T>::store(y, c, mt::silu_as<T>(v0) * v1);
  else if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float2*>(y + 2 * c) = make_float2(v0, v1);
  else
    *reinterpret_cast<uint32_t*>(y + 2 * c) = bf16x2_pack(v0, v1);
}

// One launch for NT <= ONE_TOKENS tokens with at most ONE_LOW low products in
// all: 16 rows of W (GU: 8 gate rows and their 8 up rows), a row a wave, as dot
// products with every token; the low products, a row of A_a each, are dealt to
// the same waves.  Whole rows by neighbouring lanes, and up to d_in = 2048 all
// loads of a wave at once.
constexpr int ONE_TOKENS = 4, ONE_LOW = 64, ONE_WAVES = 16;

template <typename T, int NT, bool GU>
__global__ __launch_bounds__(MOELB_WAVE * ONE_WAVES) void adapter_one_kernel(AdapterArgs p) {
  __shared__ float base[16][NT];
  __shared__ float low[ONE_LOW];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int out = GU ? p.d_out / 2 : p.d_out;
  const int n0 = block_of(p) * (GU ? 8 : 16);
  auto wrow = [&](int i) {  // row of W for row i of the workgroup
    const int c = n0 + (GU ? i & 7 : i);
    return (c < out ? c : 0) + (GU && i >= 8 ? out : 0);
  };
  const T* x = static_cast<const T*>(p.x);
  const T* w = static_cast<const T*>(p.w) + (size_t)wrow(wave) * p.d_in;
  // the output of this thread: token, row (GU: gate row and its up row)
  const int rows = GU ? 8 : 16;
  const int tt = threadIdx.x / rows, tj = threadIdx.x % rows;
  const bool mine = tt < p.Ttok && n0 + tj < out;
  const int own = mine ? id_of(p, tt) : -1;
  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.f;
#pragma unroll 4
  for (int k = lane * 8; k < p.d_in; k += MOELB_WAVE * 8) {
    float a[8];
    load_vec(w + k, a);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float v[8];
      load_vec(x + (size_t)min(t, p.Ttok - 1) * p.d_in + k, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[t] = fmaf(a[q], v[q], acc[t]);
    }
  }
  const int nlow = p.n > 0 ? p.Ttok * p.r : 0;
  for (int i = wave; i < nlow; i += ONE_WAVES) {
    const int t = i / p.r, id = __builtin_amdgcn_readfirstlane(id_of(p, t));
    if (id < 0) continue;
    const T* a = static_cast<const T*>(p.a) + ((size_t)id * p.r + i % p.r) * p.d_in;
    float v = 0.f;
#pragma unroll 4
    for (int k = lane * 8; k < p.d_in; k += MOELB_WAVE * 8) {
      float u[8], s[8];
      load_vec(a + k, u);
      load_vec(x + (size_t)t * p.d_in + k, s);
#pragma unroll
      for (int q = 0; q < 8; ++q) v = fmaf(u[q], s[q], v);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, MOELB_WAVE);
    if (lane == 0) low[i] = v * p.scale[id];
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[t] += __shfl_xor(acc[t], o, MOELB_WAVE);
    if (lane == 0) base[wave][t] = acc[t];
  }
  // the first 16 ranks of this thread's B rows, on their way while the sums meet
  const T* b0 = static_cast<const T*>(p.b) + ((size_t)max(own, 0) * p.d_out + wrow(tj)) * p.r;
  const T* b1 = static_cast<const T*>(p.b) + ((size_t)max(own, 0) * p.d_out + wrow(tj + 8)) * p.r;
  float u0[2][8], u1[2][8];
  if (own >= 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_vec(b0 + min(h * 8, p.r - 8), u0[h]);
      if (GU) load_vec(b1 + min(h * 8, p.r - 8), u1[h]);
    }
  }
  __syncthreads();
  if (!mine) return;
  float v0 = base[tj][tt], v1 = GU ? base[tj + 8][tt] : 0.f;
  if (own >= 0) {
    const float* l = low + tt * p.r;
    for (int k = 0; k < p.r; k += 8) {
      if (k >= 16) {
        load_vec(b0 + k, u0[0]);
        if (GU) load_vec(b1 + k, u1[0]);
      }
      const bool h = k == 8;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v0 = fmaf(l[k + q], h ? u0[1][q] : u0[0][q], v0);
        if (GU) v1 = fmaf(l[k + q], h ? u1[1][q] : u1[0][q], v1);
      }
    }
  }
  if (GU) v0 = mt::silu_as<T>(v0) * v1;
  Elem<T>::store(static_cast<T*>(p.y), (size_t)tt * out + n0 + tj, v0);
}

// ---------------------------------------------------------------- host

// Few tokens' kernels up to here: 64-token blocks re-read W, from the caches
// (d = 4096: 200 tokens 33 us against 47 on the tile, 400 tokens 54 against 52).
constexpr int FEW_TOKENS = 256;

// `blocks` workgroups in launches of less than 2^32 threads, each told the
// number of its first.
int launch_blocks(void (*kernel)(AdapterArgs), size_t blocks, unsigned threads, AdapterArgs p, hipStream_t s) {
  if (blocks > 0x7fffffffull) return MOELB_EINVAL;
  const size_t most = moelb_most_blocks(threads) & ~(size_t)7;
  for (size_t b = 0; b < blocks; b += most) {
    p.first = (int)b;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(threads), 0, s, p);
    MOELB_CHECK_LAUNCH();
  }
  return MOELB_OK;
}

template <int F, bool GU>
int launch_tile(AdapterArgs p, hipStream_t s) {
  const int B = 64 * F, bn = GU ? B / 2 : B, out = GU ? p.d_out / 2 : p.d_out;
  p.ntn = (out + bn - 1) / bn;
  const size_t grid = ((size_t)((p.Ttok + B - 1) / B) * p.ntn + 7) / 8 * 8;
  if (grid > moelb_most_blocks(mt::THREADS)) return MOELB_EINVAL;
  if (!moelb_allow_lds(adapter_tile_kernel<F, GU>, mt::lds_bytes<F>())) return MOELB_ELAUNCH;
  hipLaunchKernelGGL((adapter_tile_kernel<F, GU>), dim3((unsigned)grid, p.splits), dim3(mt::THREADS), mt::lds_bytes<F>(),
                     s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

// Parts of k for few tokens: about a workgroup a compute unit, at least 256 wide
// (twice as many cost more in partial sums than they gain).
int few_splits(int T, int d_in, int d_out) {
  const int blocks = (d_out + 63) / 64 * ((T + 63) / 64), want = 256 / blocks, most = d_in / 256;
  const int s = want < most ? want : most;
  return s < 1 ? 1 : s > 16 ? 16 : s;
}

// Parts of k for the 128-row tiles of prompts: two workgroups a compute unit,
// at least 512 wide.  1: whole sums, no partial ones.
int tile_splits(int T, int d_in, int d_out) {
  const size_t tiles = (size_t)((T + 127) / 128) * ((d_out + 127) / 128);
  const size_t want = 512 / tiles, most = (size_t)d_in / 512;
  const size_t s = want < most ? want : most;
  return s < 1 ? 1 : s > 8 ? 8 : (int)s;
}

// Likewise for the low products of prompts.
int low_splits(int T, int d_in) {
  const int blocks = (T + LOW_TOK - 1) / LOW_TOK, want = 512 / blocks, most = d_in / 256;
  const int s = want < most ? want : most;
  return s < 1 ? 1 : s > 16 ? 16 : s;
}

bool one_launch(int T, int n, int r) { return T <= ONE_TOKENS && (n == 0 || T * r <= ONE_LOW); }

template <typename T, int NT, bool GU>
int launch_one(const AdapterArgs& p, hipStream_t s) {
  const int out = GU ? p.d_out / 2 : p.d_out, rows = GU ? 8 : 16;
  return launch_blocks(adapter_one_kernel<T, NT, GU>, (out + rows - 1) / rows, MOELB_WAVE * ONE_WAVES, p, s);
}

template <typename T, bool GU>
int launch_sum(const AdapterArgs& p, hipStream_t s) {
  return launch_blocks(adapter_few_sum_kernel<T, GU>, ((size_t)p.Ttok * (p.d_out / 2) + 255) / 256, 256, p, s);
}

template <typename T, bool GU>
int launch_ones(const AdapterArgs& p, hipStream_t s) {
  return p.Ttok == 1   ? launch_one<T, 1, GU>(p, s)
         : p.Ttok == 2 ? launch_one<T, 2, GU>(p, s)
                       : launch_one<T, 4, GU>(p, s);
}

template <bool GU>
int launch_few(AdapterArgs p, hipStream_t s) {
  if (one_launch(p.Ttok, p.n, p.r)) return launch_ones<uint16_t, GU>(p, s);
  p.splits = few_splits(p.Ttok, p.d_in, p.d_out);
  const int tok = p.Ttok <= 16 ? 16 : p.Ttok <= 32 ? 32 : 64;
  p.nbase = (p.d_out + 63) / 64 * p.splits * ((p.Ttok + tok - 1) / tok);
  const size_t grid = (size_t)p.nbase + (p.n > 0 ? (p.Ttok * p.r + 3) / 4 : 0);
  const int st = launch_blocks(p.Ttok <= 16   ? adapter_few_kernel<1>
                               : p.Ttok <= 32 ? adapter_few_kernel<2>
                                              : adapter_few_kernel<4>,
                               grid, 256, p, s);
  if (st != MOELB_OK) return st;
  return launch_sum<uint16_t, GU>(p, s);
}

template <bool GU>
int launch_prompts(AdapterArgs p, hipStream_t s) {
  if (p.n > 0) {
    p.splits = low_splits(p.Ttok, p.d_in);
    if (!moelb_allow_lds(adapter_low_tile_kernel, mt::lds_bytes<2>())) return MOELB_ELAUNCH;
    hipLaunchKernelGGL(adapter_low_tile_kernel, dim3((p.Ttok + LOW_TOK - 1) / LOW_TOK, p.splits, (p.r + 63) / 64),
                       dim3(256), mt::lds_bytes<2>(), s, p);
    MOELB_CHECK_LAUNCH();
    const long long threads = (long long)p.Ttok * (p.r / 4);
    hipLaunchKernelGGL(adapter_low_sum_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, p);
    MOELB_CHECK_LAUNCH();
  }
  if (mt::large_tiles((size_t)((p.Ttok + 255) / 256) * ((p.d_out + 255) / 256),
                      (size_t)((p.Ttok + 127) / 128) * ((p.d_out + 127) / 128))) {
    p.splits = 1;
    return launch_tile<4, GU>(p, s);
  }
  p.splits = tile_splits(p.Ttok, p.d_in, p.d_out);
  const int st = launch_tile<2, GU>(p, s);
  if (st != MOELB_OK || p.splits == 1) return st;
  p.n = 0;  // the adapters are in the partial sums
  return launch_sum<uint16_t, GU>(p, s);
}

// fp32: parts of k of the 64 x 64 tiles, about a workgroup a compute unit, at
// least 256 wide (64 tokens, 3088 x 1248, no adapters: 16 us against 70 whole).
int f32_splits(int T, int d_in, int d_out) {
  const size_t tiles = (size_t)((T + 63) / 64) * ((d_out + 63) / 64);
  const size_t want = 256 / tiles, most = (size_t)d_in / 256;
  const size_t s = want < most ? want : most;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}
// Few tokens: the adapters are the sum's kernel's, where a thread reads its own
// rows of B (T x d_out x r values in all).  Else the tile walks the adapters
// among its tokens, dealt over the parts of k.  3088 x 1248, r = 64, 25 adapters
// in any order: 64 tokens 25 us against 34, 128 (gated) 38 against 41, but with
// 8 runs of one adapter 37 against 33.  64 tokens, 1024 x 8192, r = 256 (134 M
// values): 119 against 106, in runs 96 against 57.
constexpr int F32_FEW_TOKENS = 128;
constexpr size_t F32_FEW_VALUES = (size_t)16 << 20;
bool f32_few(int T, int d_out, int n, int r) {
  return n > 0 && T <= F32_FEW_TOKENS && (size_t)T * d_out * r <= F32_FEW_VALUES;
}

// Prompts' low products: four ranks a wave, which share the token's x, from here
// on (r = 64: 2687 tokens, d_in = 312, 50 us a call against 70 with one rank;
// 436 tokens, d_in = 4088, 136 against 147; 2768 tokens, d_in = 1832, 190
// against 179); below, a rank a wave fills the compute units.
constexpr size_t F32_FOUR_RANKS = 16384;

template <bool GU>
int launch_f32(AdapterArgs p, hipStream_t s) {
  if (one_launch(p.Ttok, p.n, p.r)) return launch_ones<float, GU>(p, s);
  const bool few = f32_few(p.Ttok, p.d_out, p.n, p.r);
  if (!few && p.n > 0) {
    const size_t waves = (size_t)p.Ttok * p.r;
    const bool four = waves >= F32_FOUR_RANKS;
    const size_t blocks = four ? (waves / 4 + 3) / 4 : (waves + 3) / 4;
    const int st =
        launch_blocks(four ? adapter_low_rows_f32_kernel<4> : adapter_low_rows_f32_kernel<1>, blocks, 256, p, s);
    if (st != MOELB_OK) return st;
  }
  const int bn = GU ? 32 : 64, out = GU ? p.d_out / 2 : p.d_out;
  p.ntn = (out + bn - 1) / bn;
  p.splits = f32_splits(p.Ttok, p.d_in, p.d_out);
  const size_t base = ((size_t)((p.Ttok + 63) / 64) * p.ntn + 7) / 8 * 8 * p.splits;
  constexpr int waves = mt::S_THREADS / MOELB_WAVE;
  const size_t grid = base + (few && p.n > 0 ? (p.Ttok * p.r + waves - 1) / waves : 0);
  if (grid > 0x7fffffffull) return MOELB_EINVAL;
  p.nbase = (int)base;
  const int st = launch_blocks(few ? adapter_tile_f32_kernel<GU, true> : adapter_tile_f32_kernel<GU, false>, grid,
                               mt::S_THREADS, p, s);
  if (st != MOELB_OK) return st;
  if (!few && p.splits == 1) return MOELB_OK;
  if (!few) p.n = 0;  // the adapters are in the partial sums
  return launch_sum<float, GU>(p, s);
}

}  // namespace

extern "C" size_t moelb_adapter_projection_workspace_bytes(int T, int d_in, int d_out, int n, int r, int dtype) {
  if (T < 0 || d_in < 1 || d_out < 1 || n < 0 || r < 0 || !moelb_dtype_ok(dtype)) return 0;
  const bool bf = dtype == MOELB_BF16, few = bf ? T <= FEW_TOKENS : f32_few(T, d_out, n, r);
  if (T == 0 || one_launch(T, n, r)) return 0;
  // low, and behind it the partial sums of few tokens, or of low itself
  const size_t low = n > 0 ? moelb_align256((size_t)T * r * (few ? 4 : moelb_elem_bytes(dtype))) : 0;
  if (few) return low + (size_t)(bf ? few_splits(T, d_in, d_out) : f32_splits(T, d_in, d_out)) * T * d_out * 4;
  const size_t lows = bf && n > 0 ? (size_t)low_splits(T, d_in) * T * r * 4 : 0;
  const int ts = bf ? tile_splits(T, d_in, d_out) : f32_splits(T, d_in, d_out);
  const size_t sums = ts > 1 ? (size_t)ts * T * d_out * 4 : 0;  // after low's own are added
  return low + (lows > sums ? lows : sums);
}

extern "C" int moelb_adapter_projection(const void* x, int T, int d_in, int d_out, int dtype, const void* w,
                                        const int32_t* ids, const void* a, const void* b, const float* scale, int n,
                                        int r, int gated, void* ws, size_t ws_bytes, void* y, void* stream) {
  if (T < 0 || d_in <= 0 || d_in % 8 != 0 || d_out <= 0 || d_out % (gated ? 16 : 8) != 0 || !moelb_dtype_ok(dtype))
    return MOELB_EINVAL;
  if (n < 0 || (n > 0 && (r < 8 || r > 256 || r % 8 != 0))) return MOELB_EINVAL;
  if (!w || (n > 0 && (!a || !b || !scale)) || (T > 0 && (!x || !y || (n > 0 && !ids)))) return MOELB_EINVAL;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(a) |
       reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(y)) & 15)
    return MOELB_EINVAL;
  const size_t eb = moelb_elem_bytes(dtype), most = mt::MAX_BYTES;
  if ((size_t)T * d_in * eb >= most || (size_t)d_out * d_in * eb >= most ||
      (n > 0 && ((size_t)n * d_out * r * eb >= most || (size_t)T * r * eb >= most || (size_t)r * d_in * eb >= most)))
    return MOELB_EINVAL;
  const size_t need = moelb_adapter_projection_workspace_bytes(T, d_in, d_out, n, r, dtype);
  if (need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < need)) return MOELB_EWORKSPACE;
  if (T == 0) return MOELB_OK;
  const bool bf = dtype == MOELB_BF16;
  const size_t low = n > 0 ? moelb_align256((size_t)T * r * (bf && T <= FEW_TOKENS ? 4 : eb)) : 0;
  AdapterArgs p = {};
  p.x = x, p.w = w, p.ids = ids, p.a = a, p.b = b, p.scale = scale, p.low = ws;
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + low);
  p.y = y;
  p.Ttok = T, p.d_in = d_in, p.d_out = d_out, p.n = n, p.r = n > 0 ? r : 8;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (bf) {
    if (T <= FEW_TOKENS) return gated ? launch_few<true>(p, s) : launch_few<false>(p, s);
    return gated ? launch_prompts<true>(p, s) : launch_prompts<false>(p, s);
  }
  return gated ? launch_f32<true>(p, s) : launch_f32<false>(p, s);
}
