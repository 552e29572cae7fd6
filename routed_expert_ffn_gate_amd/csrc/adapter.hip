// A shared projection with the low-rank adapters of many requests beside it.
//
//   y[t] = x[t] W^T + scale_a (x[t] A_a^T) B_a^T,  a = ids[t]
// (no second term for a token without an adapter), optionally gated: W and B_a
// hold gate rows and then up rows, y = silu(gate) * up.  It stands where the
// layer's always-on shared expert stands, whose projections every request
// shares while its adapter is the request's own.
//
// Two launches.  The first forms low[t] = scale_a x[t] A_a^T (r values a
// token, in the storage type: an operand of the second product, off by half a
// step of the adapter's small share of y).  The second is the projection, with
// the adapters inside its sum:
//  * Prompts (adapter_tile_kernel): the product x W^T on the tile of
//    mfma_tile.h.  Then, into the same accumulators, low B_a^T for every adapter
//    that occurs among a wave's rows, fragments straight from memory (r values
//    a row: they sit in L2).  An accumulator lane belongs to one token, so a
//    lane whose token has another adapter keeps its old value: nothing of one
//    request's adapter, NaN or infinity included, reaches another's tokens.
//    Rows of one request take one such product; mixed rows take one for each
//    adapter among them.
//  * Few tokens (adapter_few_kernel): the weights' bytes bound it, so a
//    workgroup takes 16 rows of W and 8 waves cut the sum over k between them,
//    v_mfma_f32_16x16x32_bf16 straight from registers; partial sums meet in LDS
//    in wave order, and each thread adds the rank-r product of its outputs.
#include "mfma_tile.h"

namespace {

struct AdapterArgs {
  const void* x;
  const void* w;
  const int32_t* ids;
  const void* a;
  const void* b;
  const float* scale;
  void* low;  // [T][r]
  void* y;
  int Ttok, d_in, d_out, n, r, ntn;
};

__device__ __forceinline__ uint32_t bytes32(size_t n) { return n < mt::OUTSIDE ? (uint32_t)n : mt::OUTSIDE; }
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

// A wave per (token, rank): a dot product over d_in, 8 values a lane and step.
template <typename T>
__global__ __launch_bounds__(256) void adapter_low_rows_kernel(AdapterArgs p) {
  const long long wv = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int t = (int)(wv / p.r), rr = (int)(wv % p.r);
  if (t >= p.Ttok) return;
  const int id = id_of(p, t);
  if (id < 0) return;
  const T* x = static_cast<const T*>(p.x) + (size_t)t * p.d_in;
  const T* a = static_cast<const T*>(p.a) + ((size_t)id * p.r + rr) * p.d_in;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int k = lane * 8; k < p.d_in; k += MOELB_WAVE * 8) {
    float u[8], v[8];
    load_vec(x + k, u);
    load_vec(a + k, v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 = fmaf(u[i], v[i], s0);
      s1 = fmaf(u[i + 1], v[i + 1], s1);
    }
  }
  s0 += s1;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s0 += __shfl_xor(s0, o, MOELB_WAVE);
  if (lane == 0) Elem<T>::store(static_cast<T*>(p.low), (size_t)t * p.r + rr, s0 * p.scale[id]);
}

// 32 tokens x 64 ranks of the blockIdx.y-th adapter among the tile's tokens;
// 8 waves cut the sum over k, partial sums meet in LDS in wave order.  Rows of
// tokens with another adapter are formed and dropped: tokens of a request are
// neighbours, so a tile has one or two adapters.
constexpr int LOW_TOK = 32, LOW_WAVES = 8;

__global__ __launch_bounds__(MOELB_WAVE * LOW_WAVES) void adapter_low_tile_kernel(AdapterArgs p) {
  __shared__ float part[LOW_WAVES][LOW_TOK * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.x * LOW_TOK, r0 = blockIdx.z * 64;
  const int mine = t0 + (lane & 31) < p.Ttok ? id_of(p, t0 + (lane & 31)) : -1;
  uint64_t left = __ballot(mine >= 0);
  int id = -1;
  for (int i = 0; i <= (int)blockIdx.y; ++i) {  // the blockIdx.y-th distinct id, in token order
    if (!left) return;
    id = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    left &= ~__ballot(mine == id);
  }
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  const uint16_t* a = static_cast<const uint16_t*>(p.a) + (size_t)id * p.r * p.d_in;
  const int steps = (p.d_in + 15) / 16, per = (steps + LOW_WAVES - 1) / LOW_WAVES;
  const int k0 = wave * per * 16, k1 = min(p.d_in, k0 + per * 16);
  const uint16_t* xr = x + (size_t)min(t0 + (lane & 31), p.Ttok - 1) * p.d_in + (lane >> 5) * 8;
  const uint16_t* ar[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    ar[i] = a + (size_t)min(r0 + i * 32 + (lane & 31), p.r - 1) * p.d_in + (lane >> 5) * 8;
  f32x16_t acc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[i][q] = 0.f;
  const bool two = p.r - r0 > 32;
  const int kc = (lane >> 5) * 8;
  for (int k = k0; k < k1; k += 64) {  // four steps' loads in flight
    bf16x8_t fx[4], f0[4], f1[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      fx[u] = frag_at(xr, k + u * 16, kc, k1);
      f0[u] = frag_at(ar[0], k + u * 16, kc, k1);
      if (two) f1[u] = frag_at(ar[1], k + u * 16, kc, k1);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f0[u], fx[u], acc[0], 0, 0, 0);
      if (two) acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f1[u], fx[u], acc[1], 0, 0, 0);
    }
  }
  // lane: token lane % 32; element j: rank (j / 4) * 8 + (lane / 32) * 4 + j % 4
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4_t v = {acc[i][q * 4], acc[i][q * 4 + 1], acc[i][q * 4 + 2], acc[i][q * 4 + 3]};
      const int c4 = i * 8 + q * 2 + (lane >> 5);
      *reinterpret_cast<f32x4_t*>(&part[wave][(lane & 31) * 64 + ((c4 ^ (lane & 15)) * 4)]) = v;
    }
  __syncthreads();
  const int tok = threadIdx.x >> 4, c4 = threadIdx.x & 15;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < LOW_WAVES; ++w)
    v += *reinterpret_cast<const f32x4_t*>(&part[w][tok * 64 + ((c4 ^ (tok & 15)) * 4)]);
  const int t = t0 + tok, rr = r0 + c4 * 4;
  if (t >= p.Ttok || rr >= p.r || id_of(p, t) != id) return;
  const float s = p.scale[id];
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.low) + (size_t)t * p.r + rr) =
      make_uint2(bf16x2_pack(v[0] * s, v[1] * s), bf16x2_pack(v[2] * s, v[3] * s));
}

// ---------------------------------------------------------------- prompts

// acc += low B^T for the adapters among this wave's 32 F rows.  own[mi]: the
// adapter of row block mi's lane % 32-th token, -1: none.  brow(ni): row of B
// for this lane in column block ni.
template <int F, class Row>
__device__ __forceinline__ void add_adapters(const AdapterArgs& p, const uint16_t* const (&low)[F],
                                             const int (&own)[F], Row brow, f32x16_t (&acc)[F][F]) {
  const int kc = ((threadIdx.x & 63) >> 5) * 8;
  int left[F];
#pragma unroll
  for (int mi = 0; mi < F; ++mi) left[mi] = own[mi];
  for (;;) {
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

__device__ __forceinline__ void store_gated(uint16_t* y, const float* g, const float* u) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = silu_f32(g[i]) * u[i];
  mt::store8(y, v);
}
__device__ __forceinline__ void store_gated(float* y, const float* g, const float* u) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = silu_f32(g[i]) * u[i];
  mt::store8(y, v);
}

// Tile order: as the grouped FFN's, 8 token tiles x every column tile, dealt in
// contiguous ranges to the 8 XCDs.
__device__ __forceinline__ bool tile_of(const AdapterArgs& p, int B, int& mi, int& ni) {
  const int ntm = (p.Ttok + B - 1) / B, total = ntm * p.ntn;
  const int per = (total + 7) / 8;
  const int t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || t >= total) return false;
  const int group = t / (8 * p.ntn), gm = min(8, ntm - group * 8), local = t - group * 8 * p.ntn;
  ni = local / gm;
  mi = group * 8 + local % gm;
  return true;
}

template <int F, bool GU>
__global__ __launch_bounds__(mt::THREADS) void adapter_tile_kernel(AdapterArgs p) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  constexpr int B = 64 * F;
  int mi, ni;
  if (!tile_of(p, B, mi, ni)) return;
  const int t0 = mi * B, n0 = ni * (GU ? B / 2 : B);
  const int out = GU ? p.d_out / 2 : p.d_out;
  auto trow = [&](int i) { return min(t0 + i, p.Ttok - 1); };
  auto wrow = [&](int i) {
    const int c = n0 + (GU ? i % (B / 2) : i);
    return (c < out ? c : 0) + (GU && i >= B / 2 ? out : 0);
  };
  mt::RowOp<F> oa, ob;
  oa.init(p.x, bytes32((size_t)p.Ttok * p.d_in * 2), p.d_in, p.d_in, trow);
  ob.init(p.w, bytes32((size_t)p.d_out * p.d_in * 2), p.d_in, p.d_in, wrow);
  f32x16_t acc[F][F];
  mt::k_loop<F, GU>(lds, oa, ob, (p.d_in + mt::BK - 1) / mt::BK, acc);
  if (p.n > 0) {
    const int lane = threadIdx.x & 63, wm = threadIdx.x >> 7, wn = (threadIdx.x >> 6) & 1;
    const uint16_t* low[F];
    int own[F];
#pragma unroll
    for (int mi = 0; mi < F; ++mi) {
      const int t = t0 + wm * 32 * F + mi * 32 + (lane & 31);
      own[mi] = t < p.Ttok ? id_of(p, t) : -1;
      low[mi] = static_cast<const uint16_t*>(p.low) + (size_t)min(t, p.Ttok - 1) * p.r + (lane >> 5) * 8;
    }
    add_adapters<F>(p, low, own, [&](int ni) { return wrow(mt::block_col<F, GU>(wn, ni) + (lane & 31)); }, acc);
  }
  uint16_t* y = static_cast<uint16_t*>(p.y);
  if constexpr (GU) {
    mt::drain<F, true>(lds, acc, [&](int r, int c, const float* g, const float* u) {
      if (t0 + r < p.Ttok && n0 + c < out) store_gated(y + (size_t)(t0 + r) * out + n0 + c, g, u);
    });
  } else {
    mt::drain<F, false>(lds, acc, [&](int r, int c, const float* v) {
      if (t0 + r < p.Ttok && n0 + c < out) mt::store8(y + (size_t)(t0 + r) * out + n0 + c, v);
    });
  }
}

// fp32: the same sum on 64 x 64 tiles.
template <bool GU>
__global__ __launch_bounds__(mt::THREADS) void adapter_tile_f32_kernel(AdapterArgs p) {
  __shared__ __align__(16) float lds[mt::S_FLOATS];
  __shared__ int tok[64];
  int mi, ni;
  if (!tile_of(p, 64, mi, ni)) return;
  const int t0 = mi * 64, n0 = ni * (GU ? 32 : 64);
  const int out = GU ? p.d_out / 2 : p.d_out;
  const float* x = static_cast<const float*>(p.x);
  const float* w = static_cast<const float*>(p.w);
  const float* low = static_cast<const float*>(p.low);
  auto wrow = [&](int i) {
    const int c = n0 + (GU ? i & 31 : i);
    return c < out ? c + (GU && i >= 32 ? out : 0) : -1;
  };
  f32x16_t acc;
  {
    auto pa = [&](int i, int k) { return t0 + i < p.Ttok ? x + (size_t)(t0 + i) * p.d_in + k : nullptr; };
    auto pb = [&](int i, int k) { return wrow(i) >= 0 ? w + (size_t)wrow(i) * p.d_in + k : nullptr; };
    mt::k_loop_f32<false, false>(lds, pa, pb, p.d_in, acc);
  }
  if (p.n > 0) {
    // every wave walks the tile's adapters (they load the rows together); a
    // lane whose token has another one keeps its value
    if (threadIdx.x < 64) tok[threadIdx.x] = t0 + (int)threadIdx.x < p.Ttok ? id_of(p, t0 + threadIdx.x) : -1;
    __syncthreads();
    int left = tok[threadIdx.x & 63];
    const int own = tok[(threadIdx.x >> 7) * 32 + (threadIdx.x & 31)];
    const int ti = threadIdx.x >> 2;  // the row this thread fetches
    for (uint64_t some = __ballot(left >= 0); some; some = __ballot(left >= 0)) {
      const int id = __builtin_amdgcn_readlane(left, __builtin_ctzll(some));
      if (left == id) left = -1;
      const float* b = static_cast<const float*>(p.b) + (size_t)id * p.d_out * p.r;
      auto pa = [&](int, int k) { return tok[ti] == id ? low + (size_t)(t0 + ti) * p.r + k : nullptr; };
      auto pb = [&](int i, int k) { return wrow(i) >= 0 ? b + (size_t)wrow(i) * p.r + k : nullptr; };
      f32x16_t more;
      __syncthreads();
      mt::k_loop_f32<false, false>(lds, pa, pb, p.r, more);
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[q] = own == id ? acc[q] + more[q] : acc[q];
    }
  }
  float* y = static_cast<float*>(p.y);
  if constexpr (GU) {
    mt::drain_f32<true>(lds, acc, [&](int r, int c, const float* g, const float* u) {
      if (t0 + r < p.Ttok && n0 + c < out) store_gated(y + (size_t)(t0 + r) * out + n0 + c, g, u);
    });
  } else {
    mt::drain_f32<false>(lds, acc, [&](int r, int c, const float* v) {
      if (t0 + r < p.Ttok && n0 + c < out) mt::store8(y + (size_t)(t0 + r) * out + n0 + c, v);
    });
  }
}

// ---------------------------------------------------------------- few tokens

// 16 rows of W (GU: 8 gate rows and their 8 up rows) x 16 NB tokens
// (blockIdx.y: which 16 NB).  8 waves cut k; each lane holds row (or token)
// lane % 16 and k (lane / 16) * 8 .. of a 32-wide step.
constexpr int FEW_WAVES = 8;

template <int NB, bool GU>
__global__ __launch_bounds__(MOELB_WAVE * FEW_WAVES) void adapter_few_kernel(AdapterArgs p) {
  constexpr int TOK = 16 * NB;
  __shared__ f32x4_t part[FEW_WAVES][TOK * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int out = GU ? p.d_out / 2 : p.d_out;
  const int n0 = blockIdx.x * (GU ? 8 : 16), t0 = blockIdx.y * TOK;
  auto wrow = [&](int i) {  // row of W for tile row i
    const int c = n0 + (GU ? i & 7 : i);
    return (c < out ? c : 0) + (GU && i >= 8 ? out : 0);
  };
  const uint16_t* w = static_cast<const uint16_t*>(p.w) + (size_t)wrow(lane & 15) * p.d_in + (lane >> 4) * 8;
  const uint16_t* x[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
    x[i] = static_cast<const uint16_t*>(p.x) + (size_t)min(t0 + i * 16 + (lane & 15), p.Ttok - 1) * p.d_in +
           (lane >> 4) * 8;
  const int steps = (p.d_in + 31) / 32, per = (steps + FEW_WAVES - 1) / FEW_WAVES;
  const int k0 = wave * per * 32, k1 = min(p.d_in, k0 + per * 32);
  f32x4_t acc[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int kc = (lane >> 4) * 8;
  for (int k = k0; k < k1; k += 128) {  // four steps' loads in flight
    bf16x8_t fw[4], fx[4][NB];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      fw[u] = frag_at(w, k + u * 32, kc, k1);
#pragma unroll
      for (int i = 0; i < NB; ++i) fx[u][i] = frag_at(x[i], k + u * 32, kc, k1);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < NB; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fw[u], fx[u][i], acc[i], 0, 0, 0);
  }
  // lane: token lane % 16 of block i, rows (lane / 16) * 4 ..
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int tok = i * 16 + (lane & 15);
    part[wave][tok * 4 + ((lane >> 4) ^ ((tok >> 1) & 3))] = acc[i];
  }
  __syncthreads();
  // thread -> token, two rows: gate and up row j, or rows 2 j and 2 j + 1
  for (int c = threadIdx.x; c < TOK * 8; c += MOELB_WAVE * FEW_WAVES) {
    const int tok = c >> 3, j = c & 7, t = t0 + tok;
    if (t >= p.Ttok) continue;
    const int i0 = GU ? j : 2 * j, i1 = GU ? j + 8 : 2 * j + 1;
    if (n0 + (GU ? j : 2 * j) >= out) continue;
    float v0 = 0.f, v1 = 0.f;
    const int sw = (tok >> 1) & 3;
#pragma unroll
    for (int q = 0; q < FEW_WAVES; ++q) {
      const float* f = reinterpret_cast<const float*>(&part[q][tok * 4]);
      v0 += f[((i0 >> 2) ^ sw) * 4 + (i0 & 3)];
      v1 += f[((i1 >> 2) ^ sw) * 4 + (i1 & 3)];
    }
    const int id = id_of(p, t);
    if (id >= 0) {
      const uint16_t* low = static_cast<const uint16_t*>(p.low) + (size_t)t * p.r;
      const uint16_t* b = static_cast<const uint16_t*>(p.b) + (size_t)id * p.d_out * p.r;
      const uint16_t* b0 = b + (size_t)wrow(i0) * p.r;
      const uint16_t* b1 = b + (size_t)wrow(i1) * p.r;
      for (int k = 0; k < p.r; k += 8) {
        float s[8], u[8], v[8];
        load_vec(low + k, s);
        load_vec(b0 + k, u);
        load_vec(b1 + k, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v0 = fmaf(s[q], u[q], v0);
          v1 = fmaf(s[q], v[q], v1);
        }
      }
    }
    uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)t * out + n0;
    if (GU)
      y[j] = f32_to_bf16(silu_f32(v0) * v1);
    else
      *reinterpret_cast<uint32_t*>(y + 2 * j) = bf16x2_pack(v0, v1);
  }
}

// ---------------------------------------------------------------- host

constexpr int FEW_TOKENS = 64;

template <int F, bool GU>
int launch_tile(AdapterArgs p, hipStream_t s) {
  const int B = 64 * F, bn = GU ? B / 2 : B, out = GU ? p.d_out / 2 : p.d_out;
  p.ntn = (out + bn - 1) / bn;
  const size_t grid = ((size_t)((p.Ttok + B - 1) / B) * p.ntn + 7) / 8 * 8;
  if (grid > 0x7fffffffull) return MOELB_EINVAL;
  if (!moelb_allow_lds(adapter_tile_kernel<F, GU>, mt::lds_bytes<F>())) return MOELB_ELAUNCH;
  hipLaunchKernelGGL((adapter_tile_kernel<F, GU>), dim3((unsigned)grid), dim3(mt::THREADS), mt::lds_bytes<F>(), s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

template <bool GU>
int launch_f32(AdapterArgs p, hipStream_t s) {
  const int bn = GU ? 32 : 64, out = GU ? p.d_out / 2 : p.d_out;
  p.ntn = (out + bn - 1) / bn;
  const size_t grid = ((size_t)((p.Ttok + 63) / 64) * p.ntn + 7) / 8 * 8;
  if (grid > 0x7fffffffull) return MOELB_EINVAL;
  hipLaunchKernelGGL((adapter_tile_f32_kernel<GU>), dim3((unsigned)grid), dim3(mt::THREADS), 0, s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

template <int NB, bool GU>
int launch_few(const AdapterArgs& p, hipStream_t s) {
  const int out = GU ? p.d_out / 2 : p.d_out, rows = GU ? 8 : 16;
  hipLaunchKernelGGL((adapter_few_kernel<NB, GU>), dim3((out + rows - 1) / rows, (p.Ttok + 16 * NB - 1) / (16 * NB)),
                     dim3(MOELB_WAVE * FEW_WAVES), 0, s, p);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

template <bool GU>
int launch_bf16(const AdapterArgs& p, hipStream_t s) {
  if (p.Ttok <= 16) return launch_few<1, GU>(p, s);
  if (p.Ttok <= 32) return launch_few<2, GU>(p, s);
  if (p.Ttok <= FEW_TOKENS) return launch_few<4, GU>(p, s);
  const size_t tiles = (size_t)((p.Ttok + 255) / 256) * ((p.d_out + 255) / 256);
  return tiles >= 192 ? launch_tile<4, GU>(p, s) : launch_tile<2, GU>(p, s);
}

}  // namespace

extern "C" size_t moelb_adapter_projection_workspace_bytes(int T, int d_in, int d_out, int n, int r, int dtype) {
  if (T < 0 || d_in < 1 || d_out < 1 || n < 0 || r < 0 || !moelb_dtype_ok(dtype)) return 0;
  return n > 0 ? moelb_align256((size_t)T * r * moelb_elem_bytes(dtype)) : 0;
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
  const size_t eb = moelb_elem_bytes(dtype), most = (1ull << 32) - 65536;
  if ((size_t)T * d_in * eb >= most || (size_t)d_out * d_in * eb >= most ||
      (n > 0 && ((size_t)n * d_out * r * eb >= most || (size_t)T * r * eb >= most)))
    return MOELB_EINVAL;
  const size_t need = moelb_adapter_projection_workspace_bytes(T, d_in, d_out, n, r, dtype);
  if (need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) || ws_bytes < need)) return MOELB_EWORKSPACE;
  if (T == 0) return MOELB_OK;
  AdapterArgs p = {x, w, ids, a, b, scale, ws, y, T, d_in, d_out, n, n > 0 ? r : 8, 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = dtype == MOELB_BF16;
  if (n > 0) {
    if (!bf || T <= FEW_TOKENS) {
      const long long blocks = ((long long)T * r + 3) / 4;
      if (blocks > 0x7fffffffll) return MOELB_EINVAL;
      if (bf)
        hipLaunchKernelGGL(adapter_low_rows_kernel<uint16_t>, dim3((unsigned)blocks), dim3(256), 0, s, p);
      else
        hipLaunchKernelGGL(adapter_low_rows_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, s, p);
    } else {
      const int slots = n < LOW_TOK ? n : LOW_TOK;
      hipLaunchKernelGGL(adapter_low_tile_kernel, dim3((T + LOW_TOK - 1) / LOW_TOK, slots, (r + 63) / 64),
                         dim3(MOELB_WAVE * LOW_WAVES), 0, s, p);
    }
    MOELB_CHECK_LAUNCH();
  }
  if (!bf) return gated ? launch_f32<true>(p, s) : launch_f32<false>(p, s);
  return gated ? launch_bf16<true>(p, s) : launch_bf16<false>(p, s);
}
