// Training form of the grouped SwiGLU FFN: a forward that keeps its two
// projections, and the gradients.
//
// Definition (FreeBalance, "FreeBalance: Pre-Routing Online MoE Load Balancing
// via Residual Workload Prediction", section 2.1: expert_i(h), here the SwiGLU
// block of moelb_grouped_ffn), for a row x of expert e:
//   [g, u] = W13 x, a = silu(g) u, y = W2 a
// and with s = 1 / (1 + e^-g), dy the gradient of y:
//   da = W2^T dy, dg = da u s (1 + g (1 - s)), du = da g s
//   dx = W13^T [dg, du], dW13 = sum [dg, du] x^T, dW2 = sum dy a^T
// the sums over the expert's rows.
//
// Six products, all on the tile of mfma_tile.h, over the row schedule of the
// forward (rows expert-major, "virtual" rows):
//   up     x rows (gathered) x W13, z = [g, u] kept in fp32, a out
//   down   a x W2, y rows scattered
//   da     dy rows (gathered) x W2 read as columns; the epilogue reads z and
//          writes [dg, du] and a again (a is not kept between the calls: it
//          costs one fused recomputation and saves rows x inter of memory)
//   dx     [dg, du] x W13 read as columns, dx rows scattered
//   dW13   [dg, du] and x (gathered), both read as columns, summed over rows
//   dW2    dy (gathered) and a, likewise
// z stays fp32: dg is a difference of terms in g where silu' is near 0, and a
// z of 11 bits with a scale per 64 columns lost single elements there while a
// whole step took the same time.  a and [dg, du] are rounded to the storage type,
// once each, because they are the next products' operands.
// Weight gradients: one workgroup owns a tile of one expert's gradient and
// walks that expert's rows in order, so a gradient is one fixed sum; where
// that leaves compute units idle the rows are cut into `splits` parts with
// fp32 partial sums, added in order by a second kernel.
//
// What bounds it: large groups, the matrix units at the clock they leave (busy
// 0.6 to 0.7 at 1.5 to 1.7 GHz; da 0.4 to 0.5, whose epilogue reads z and
// writes two operands); few rows a group, the weights and their gradients, at a
// third to half of the memory's rate, since a 128-row tile mostly repeats rows
// and a weight gradient's tile is one K step between its first loads and its
// stores (128 experts of 11 to 63 rows, d = 2048, inter = 768: up 227 us for 0.42
// GB read, the gradients 610 us for 1.7 GB); small calls, one launch after
// another (5 to 47 us each).  64 groups of 2048 rows, d = 2048, inter = 1024,
// bf16: forward 1.69 ms (977 TFLOP/s), backward 3.41 ms (967); the same rows in
// groups of 995 to 4079: 5.0 ms both (990).
#include "ffn_sched.h"
#include "mfma_tile.h"

namespace {

enum { OP_UP = 0, OP_DOWN = 1, OP_DA = 2, OP_DX = 3, OP_DW13 = 4, OP_DW2 = 5 };

template <typename T>
struct TrainArgs {
  const T* x;
  int rows_x;
  const T* w13;
  const T* w2;
  const T* dy;
  float* z;    // [rows][2 inter], virtual rows
  T* a;        // [rows][inter], virtual rows
  T* dz;       // [rows][2 inter], virtual rows
  T* out;      // y or dx, physical rows; dW13 or dW2
  float* part; // weight gradients: [splits][E][M][N] partial sums
  int splits;
  int chunks;  // weight gradients: units an expert's tiles are cut into
  int rows, d, inter, E, ntn, ntm;
  FfnSched s;
};

__device__ __forceinline__ uint32_t bytes_u32(size_t n) {
  return n < mt::MAX_BYTES ? (uint32_t)n : (uint32_t)mt::MAX_BYTES;
}

__device__ __forceinline__ int clampi(int v, int n) { return min(max(v, 0), n - 1); }

// The epilogues of the row-tiled products, on 8 adjacent columns at n of
// virtual row v.
template <typename T>
__device__ __forceinline__ void put_up(const TrainArgs<T>& p, int v, int n, const float* g, const float* u) {
  float* z = p.z + (size_t)v * 2 * p.inter + n;
  mt::store8(z, g);
  mt::store8(z + p.inter, u);
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = mt::silu_as<T>(g[i]) * u[i];
  mt::store8(p.a + (size_t)v * p.inter + n, a);
}

template <typename T>
__device__ __forceinline__ void put_da(const TrainArgs<T>& p, int v, int n, const float* da) {
  const float* z = p.z + (size_t)v * 2 * p.inter + n;
  float g[8], u[8], dg[8], du[8], a[8];
  mt::load8(z, g);
  mt::load8(z + p.inter, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float s, c;
    mt::sigmoid_as<T>(g[i], s, c);
    const float gs = g[i] * s;
    a[i] = gs * u[i];
    du[i] = da[i] * gs;
    dg[i] = da[i] * u[i] * (s * (1.0f + g[i] * c));
  }
  T* dz = p.dz + (size_t)v * 2 * p.inter + n;
  mt::store8(dz, dg);
  mt::store8(dz + p.inter, du);
  mt::store8(p.a + (size_t)v * p.inter + n, a);
}

// ---------------------------------------------------------------- row-tiled products

// Workgroup `block` of the product OP.
template <int F, int OP>
__device__ __forceinline__ void rows_tile(const TrainArgs<uint16_t>& p, int block, uint16_t* lds) {
  const int n_mtiles = *p.s.n_mtiles;
  const int tile = xcd_tile(block, n_mtiles * p.ntn);
  if (tile < 0) return;
  int mti, nt;
  grouped_tile(tile, n_mtiles, p.ntn, mti, nt);
  const int e = p.s.mt_e[mti], v0 = p.s.mt_v0[mti], vend = p.s.eoff[e + 1];
  const int d = p.d, I = p.inter;
  constexpr bool GU = OP == OP_UP;
  constexpr int HB = 32 * F;  // gate (or up) rows of an "up" tile
  const int n0 = nt * (GU ? HB : 64 * F);
  const int N = (OP == OP_UP || OP == OP_DA) ? I : d;
  const int K = OP == OP_DOWN ? I : OP == OP_DX ? 2 * I : d;

  mt::RowOp<F> oa;
  {
    const uint16_t* base = OP == OP_UP ? p.x : OP == OP_DOWN ? p.a : OP == OP_DA ? p.dy : p.dz;
    const int rows = OP == OP_UP ? p.rows_x : p.rows;
    const int32_t* map = OP == OP_UP ? p.s.asrc : OP == OP_DA ? p.s.rowmap : nullptr;
    oa.init(base, bytes_u32((size_t)rows * K * 2), K, K, [&](int r) {
      int v = v0 + r;
      v = v < vend ? v : v0;
      return map ? clampi(map[v], rows) : v;
    });
  }
  f32x16_t acc[F][F];
  const int KT = (K + mt::BK - 1) / mt::BK;
  if constexpr (OP == OP_UP || OP == OP_DOWN) {
    mt::RowOp<F> ob;
    const uint16_t* w = OP == OP_UP ? p.w13 + (size_t)e * 2 * I * d : p.w2 + (size_t)e * d * I;
    ob.init(w, bytes_u32((size_t)(GU ? 2 * I : d) * K * 2), K, K, [&](int r) {
      const int c = n0 + (GU ? r % HB : r);
      return (c < N ? c : 0) + (GU && r >= HB ? I : 0);
    });
    mt::k_loop<F, GU>(lds, oa, ob, KT, acc);
  } else {
    mt::ColOp<F, false> ob;
    const uint16_t* w = OP == OP_DA ? p.w2 + (size_t)e * d * I : p.w13 + (size_t)e * 2 * I * d;
    ob.init(w, bytes_u32((size_t)K * N * 2), N, K, n0, N);
    mt::k_loop<F, GU>(lds, oa, ob, KT, acc);
  }
  if constexpr (GU) {
    mt::drain<F, true>(lds, acc, [&](int r, int c, const float* g, const float* u) {
      if (v0 + r < vend && n0 + c < N) put_up(p, v0 + r, n0 + c, g, u);
    });
  } else if constexpr (OP == OP_DA) {
    mt::drain<F, false>(lds, acc, [&](int r, int c, const float* v) {
      if (v0 + r < vend && n0 + c < N) put_da(p, v0 + r, n0 + c, v);
    });
  } else {
    mt::drain<F, false>(lds, acc, [&](int r, int c, const float* v) {
      if (v0 + r < vend && n0 + c < N)
        mt::store8(p.out + (size_t)clampi(p.s.rowmap[v0 + r], p.rows) * d + n0 + c, v);
    });
  }
}

template <int TN, int OP>
__device__ __forceinline__ void rows_tile(const TrainArgs<float>& p, int block, float* lds) {
  const int n_mtiles = *p.s.n_mtiles;
  const int tile = xcd_tile(block, n_mtiles * p.ntn);
  if (tile < 0) return;
  const int mti = tile / p.ntn, nt = tile % p.ntn;
  const int e = p.s.mt_e[mti], v0 = p.s.mt_v0[mti], vend = p.s.eoff[e + 1];
  const int d = p.d, I = p.inter;
  constexpr bool GU = OP == OP_UP;
  const int n0 = nt * (GU ? TN / 2 : TN);
  const int N = (OP == OP_UP || OP == OP_DA) ? I : d;
  const int K = OP == OP_DOWN ? I : OP == OP_DX ? 2 * I : d;
  const float* base = OP == OP_UP ? p.x : OP == OP_DOWN ? p.a : OP == OP_DA ? p.dy : p.dz;
  const int rows = OP == OP_UP ? p.rows_x : p.rows;
  const int32_t* map = OP == OP_UP ? p.s.asrc : OP == OP_DA ? p.s.rowmap : nullptr;
  __shared__ int src[mt::S_BM];  // row of the left factor, -1 past the end
  if (threadIdx.x < mt::S_BM) {
    const int v = v0 + threadIdx.x;
    src[threadIdx.x] = v < vend ? (map ? clampi(map[v], rows) : v) : -1;
  }
  __syncthreads();
  auto pa = [&](int r, int k) { return src[r] < 0 ? nullptr : base + (size_t)src[r] * K + k; };
  f32x16_t acc;
  if constexpr (OP == OP_UP || OP == OP_DOWN) {
    const float* w = OP == OP_UP ? p.w13 + (size_t)e * 2 * I * d : p.w2 + (size_t)e * d * I;
    auto pb = [&](int r, int k) {
      const int c = n0 + (GU ? r % (TN / 2) : r);
      return c < N ? w + ((size_t)c + (GU && r >= TN / 2 ? I : 0)) * K + k : nullptr;
    };
    mt::k_loop_f32<TN, false, false>(lds, pa, pb, K, acc);
  } else {
    const float* w = OP == OP_DA ? p.w2 + (size_t)e * d * I : p.w13 + (size_t)e * 2 * I * d;
    auto pb = [&](int r, int k) { return n0 + r < N ? w + (size_t)k * N + n0 + r : nullptr; };
    mt::k_loop_f32<TN, false, true>(lds, pa, pb, K, acc);
  }
  if constexpr (GU) {
    mt::drain_f32<TN, true>(lds, acc, [&](int r, int c, const float* g, const float* u) {
      if (v0 + r < vend && n0 + c < N) put_up(p, v0 + r, n0 + c, g, u);
    });
  } else if constexpr (OP == OP_DA) {
    mt::drain_f32<TN, false>(lds, acc, [&](int r, int c, const float* v) {
      if (v0 + r < vend && n0 + c < N) put_da(p, v0 + r, n0 + c, v);
    });
  } else {
    mt::drain_f32<TN, false>(lds, acc, [&](int r, int c, const float* v) {
      if (v0 + r < vend && n0 + c < N)
        mt::store8(p.out + (size_t)clampi(p.s.rowmap[v0 + r], p.rows) * d + n0 + c, v);
    });
  }
}

// ---------------------------------------------------------------- weight gradients

// Workgroup -> expert, split of its rows, tile of its gradient.  An expert's
// tiles are cut into `chunks` units; the units, most rows first, go to the 8
// XCDs in turn, and the workgroups of an XCD (every eighth) take its units one
// after another.  So the tiles running at once on an XCD share an expert's
// rows in its L2, and however uneven the experts are (all rows on a few of
// them included) the XCDs get like amounts of work.
struct WTile {
  int e, mi, ni, split, n, v0;
};
template <typename T>
__device__ __forceinline__ bool w_tile(const TrainArgs<T>& p, int block, WTile& w) {
  const int per = p.ntm * p.ntn * p.splits;
  const int u = (per + p.chunks - 1) / p.chunks;
  const int j = block >> 3;
  const int unit = (j / u) * 8 + (block & 7);
  if (unit >= p.E * p.chunks) return false;
  int t = (unit % p.chunks) * u + j % u;
  if (t >= per) return false;
  w.e = p.s.order[unit / p.chunks];
  w.split = t / (p.ntm * p.ntn);
  t -= w.split * p.ntm * p.ntn;
  grouped_tile(t, p.ntm, p.ntn, w.mi, w.ni);
  const int vb = p.s.eoff[w.e], n = p.s.eoff[w.e + 1] - vb;
  const int steps = (n + mt::BK - 1) / mt::BK;
  const int ps = (steps + p.splits - 1) / p.splits * mt::BK;  // rows of a split
  const int k0 = min(n, w.split * ps);
  w.n = min(n, k0 + ps) - k0;
  w.v0 = vb + k0;
  return true;
}

template <typename T>
__device__ __forceinline__ void put_w(const TrainArgs<T>& p, const WTile& w, int M, int N, int m, int n,
                                      const float* v) {
  if (m >= M || n >= N) return;
  const size_t at = ((size_t)w.e * M + m) * N + n;
  if (p.splits > 1)
    mt::store8(p.part + (size_t)w.split * p.E * M * N + at, v);
  else
    mt::store8(p.out + at, v);
}

// A tile of zeros, for an expert (or a split) without rows.
template <int BM, int BN, typename T>
__device__ __forceinline__ void zero_w(const TrainArgs<T>& p, const WTile& w, int M, int N) {
  const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int c = threadIdx.x; c < BM * (BN / 8); c += blockDim.x)
    put_w(p, w, M, N, w.mi * BM + c / (BN / 8), w.ni * BN + (c % (BN / 8)) * 8, v);
}

template <int F, int OP>
__device__ __forceinline__ void weights_tile(const TrainArgs<uint16_t>& p, int block, uint16_t* lds) {
  WTile w;
  if (!w_tile(p, block, w)) return;
  const int d = p.d, I = p.inter;
  const int M = OP == OP_DW13 ? 2 * I : d, N = OP == OP_DW13 ? d : I;
  if (w.n == 0) {
    zero_w<64 * F, 64 * F>(p, w, M, N);
    return;
  }
  const int m0 = w.mi * 64 * F, n0 = w.ni * 64 * F;
  const int KT = (w.n + mt::BK - 1) / mt::BK;
  f32x16_t acc[F][F];
  if constexpr (OP == OP_DW13) {
    mt::ColOp<F, false> oa;
    mt::ColOp<F, true> ob;
    oa.init(p.dz + (size_t)w.v0 * M, bytes_u32((size_t)w.n * M * 2), M, w.n, m0, M);
    ob.init(p.x, bytes_u32((size_t)p.rows_x * N * 2), N, w.n, n0, N, p.s.asrc + w.v0, p.rows_x);
    mt::k_loop<F, false>(lds, oa, ob, KT, acc);
  } else {
    mt::ColOp<F, true> oa;
    mt::ColOp<F, false> ob;
    oa.init(p.dy, bytes_u32((size_t)p.rows * M * 2), M, w.n, m0, M, p.s.rowmap + w.v0, p.rows);
    ob.init(p.a + (size_t)w.v0 * N, bytes_u32((size_t)w.n * N * 2), N, w.n, n0, N);
    mt::k_loop<F, false>(lds, oa, ob, KT, acc);
  }
  mt::drain<F, false>(lds, acc, [&](int r, int c, const float* v) { put_w(p, w, M, N, m0 + r, n0 + c, v); });
}

template <int TN, int OP>
__device__ __forceinline__ void weights_tile(const TrainArgs<float>& p, int block, float* lds) {
  WTile w;
  if (!w_tile(p, block, w)) return;
  const int d = p.d, I = p.inter;
  const int M = OP == OP_DW13 ? 2 * I : d, N = OP == OP_DW13 ? d : I;
  if (w.n == 0) {
    zero_w<mt::S_BM, TN>(p, w, M, N);
    return;
  }
  const int m0 = w.mi * 64, n0 = w.ni * TN;
  f32x16_t acc;
  auto pa = [&](int r, int k) -> const float* {
    if (m0 + r >= M) return nullptr;
    if (OP == OP_DW13) return p.dz + (size_t)(w.v0 + k) * M + m0 + r;
    return p.dy + (size_t)clampi(p.s.rowmap[w.v0 + k], p.rows) * M + m0 + r;
  };
  auto pb = [&](int r, int k) -> const float* {
    if (n0 + r >= N) return nullptr;
    if (OP == OP_DW13) return p.x + (size_t)clampi(p.s.asrc[w.v0 + k], p.rows_x) * N + n0 + r;
    return p.a + (size_t)(w.v0 + k) * N + n0 + r;
  };
  mt::k_loop_f32<TN, true, true>(lds, pa, pb, w.n, acc);
  mt::drain_f32<TN, false>(lds, acc, [&](int r, int c, const float* v) { put_w(p, w, M, N, m0 + r, n0 + c, v); });
}

// ---------------------------------------------------------------- kernels

template <int F, int OP>
__global__ __launch_bounds__(mt::THREADS) void train_rows_kernel(TrainArgs<uint16_t> p) {
  extern __shared__ __align__(16) char smem[];
  rows_tile<F, OP>(p, blockIdx.x, reinterpret_cast<uint16_t*>(smem));
}
template <int TN, int OP>
__global__ __launch_bounds__(mt::S_THREADS) void train_rows_f32_kernel(TrainArgs<float> p) {
  __shared__ __align__(16) float lds[mt::STile<TN>::FLOATS];
  rows_tile<TN, OP>(p, blockIdx.x, lds);
}

// dW13, dW2 and dx all follow from [dg, du], a and dy: one launch, so the last
// round of one product's tiles runs beside the next product's.  Each block
// range starts at a multiple of 8 (the XCD of a block is its id mod 8).
template <typename T>
struct GradArgs {
  TrainArgs<T> w13, w2, x;
  int n13, n2, nx;  // their blocks
  bool x_first;     // dx's sums are the longest: its blocks come first
};
template <int F>
__global__ __launch_bounds__(mt::THREADS) void train_grads_kernel(GradArgs<uint16_t> g) {
  extern __shared__ __align__(16) char smem[];
  uint16_t* lds = reinterpret_cast<uint16_t*>(smem);
  int b = blockIdx.x;
  const int x0 = g.x_first ? 0 : g.n13 + g.n2;
  if (b >= x0 && b < x0 + g.nx) {
    rows_tile<F, OP_DX>(g.x, b - x0, lds);
    return;
  }
  if (g.x_first) b -= g.nx;
  if (b < g.n13)
    weights_tile<F, OP_DW13>(g.w13, b, lds);
  else
    weights_tile<F, OP_DW2>(g.w2, b - g.n13, lds);
}
template <int TN>
__global__ __launch_bounds__(mt::S_THREADS) void train_grads_f32_kernel(GradArgs<float> g) {
  __shared__ __align__(16) float lds[mt::STile<TN>::FLOATS];
  int b = blockIdx.x;
  const int x0 = g.x_first ? 0 : g.n13 + g.n2;
  if (b >= x0 && b < x0 + g.nx) {
    rows_tile<TN, OP_DX>(g.x, b - x0, lds);
    return;
  }
  if (g.x_first) b -= g.nx;
  if (b < g.n13)
    weights_tile<TN, OP_DW13>(g.w13, b, lds);
  else
    weights_tile<TN, OP_DW2>(g.w2, b - g.n13, lds);
}

// out[i] = sum over splits, in order, of part[s][i]; 8 values per thread.
template <typename T>
__global__ __launch_bounds__(256) void sum_splits_kernel(const float* __restrict__ part, int splits, size_t n8,
                                                         T* __restrict__ out) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  mt::load8(part + i * 8, v);
  for (int s = 1; s < splits; ++s) {
    float u[8];
    mt::load8(part + ((size_t)s * n8 + i) * 8, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += u[j];
  }
  mt::store8(out + i * 8, v);
}

// ---------------------------------------------------------------- host

// Tile height of a call (64 F, or 64 for fp32): 256 where the experts average
// enough rows and the tiles still cover the compute units.  Routed (uneven)
// rows, a whole step in us with 128 | 256, by rows an expert: 64 experts, d = 2048,
// inter = 1024: 160: 965 | 994, 192: 1077 | 1032, 384: 1603 | 1400; 128 experts,
// inter = 768: 160: 1457 | 1389, 256: 1807 | 1692; 16 experts, where the tiles
// do not cover the units: 192: 271 | 302, 384: 400 | 445, 512: 513 | 492.
int tile_rows(int rows, int E, int d, int inter, int dtype) {
  if (dtype != MOELB_BF16) return mt::S_BM;
  const int least = d < inter ? d : inter;
  const size_t tiles = (size_t)(rows + 255) / 256 * ((least + 255) / 256);
  return (size_t)rows >= (size_t)192 * E && tiles >= 192 ? 256 : 128;
}

// Column tile: as wide as the row tile, but for fp32 half of it where a call's
// row-tiled products have fewer 64-wide tiles than compute units.
int tile_cols(int rows, int E, int d, int inter, int dtype) {
  const int b = tile_rows(rows, E, d, inter, dtype);
  if (dtype == MOELB_BF16) return b;
  const int least = d < inter ? d : inter;
  return (size_t)(rows + 63) / 64 * ((least + 63) / 64) < 256 ? 32 : 64;
}

// Parts the rows of every expert are cut into for the weight gradients: enough
// workgroups for the compute units, at least 512 rows each on average.
int weight_splits(int rows, int E, int M, int N, int b, int bn) {
  const int slots = b == 256 ? 256 : 512;
  const size_t tiles = (size_t)E * ((M + b - 1) / b) * ((N + bn - 1) / bn);
  const size_t want = slots / tiles, most = (size_t)rows / E / 512;
  const size_t s = want < most ? want : most;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

struct BackLayout {
  size_t order, dz, part13, part2, total;
};
BackLayout back_layout(int rows, int num_groups, int E, int d, int inter, int dtype) {
  BackLayout l;
  const size_t eb = moelb_elem_bytes(dtype);
  const int tile = tile_rows(rows, E, d, inter, dtype), tn = tile_cols(rows, E, d, inter, dtype);
  l.order = sched_layout(rows, num_groups, E, inter, dtype, nullptr, nullptr);  // schedule tables and a
  l.dz = l.order + moelb_align256((size_t)E * 4);
  l.part13 = l.dz + moelb_align256((size_t)rows * 2 * inter * eb);
  const size_t s13 = weight_splits(rows, E, 2 * inter, d, tile, tn),
               s2 = weight_splits(rows, E, d, inter, tile, tn);
  l.part2 = l.part13 + (s13 > 1 ? moelb_align256(s13 * E * 2 * inter * d * 4) : 0);
  l.total = l.part2 + (s2 > 1 ? moelb_align256(s2 * E * inter * d * 4) : 0);
  return l;
}

// Blocks of a row-tiled product; sets its column tiles.
template <typename T>
size_t rows_grid(TrainArgs<T>& p, int BM, int bn, int N) {
  p.ntn = (N + bn - 1) / bn;
  return ((size_t)(p.rows + BM - 1) / BM + p.E) * p.ntn + 8;
}

// Blocks of a weight gradient; sets its tiles, splits and units: about 32
// tiles a unit (the compute units of an XCD), at least 32 units in all.
template <typename T>
size_t weights_grid(TrainArgs<T>& p, int BM, int BN, int M, int N) {
  p.splits = weight_splits(p.rows, p.E, M, N, BM, BN);
  p.ntm = (M + BM - 1) / BM;
  p.ntn = (N + BN - 1) / BN;
  const int per = p.ntm * p.ntn * p.splits;
  const int c = per / 32, least = (32 + p.E - 1) / p.E;
  p.chunks = c > least ? c : least;
  if (p.chunks > per) p.chunks = per;
  const int u = (per + p.chunks - 1) / p.chunks;
  return (size_t)((p.E * p.chunks + 7) / 8) * 8 * u;
}

template <typename T, int OP>
int launch_rows(TrainArgs<T> p, int BM, int BN, hipStream_t s) {
  const size_t grid = rows_grid(p, BM, OP == OP_UP ? BN / 2 : BN, (OP == OP_UP || OP == OP_DA) ? p.inter : p.d);
  const dim3 g((unsigned)grid);
  if constexpr (sizeof(T) == 4) {
    if (BN == 64)
      hipLaunchKernelGGL((train_rows_f32_kernel<64, OP>), g, dim3(mt::S_THREADS), 0, s, p);
    else
      hipLaunchKernelGGL((train_rows_f32_kernel<32, OP>), g, dim3(mt::S_THREADS), 0, s, p);
  } else if (BM == 256) {
    if (!moelb_allow_lds(train_rows_kernel<4, OP>, mt::lds_bytes<4>())) return MOELB_ELAUNCH;
    hipLaunchKernelGGL((train_rows_kernel<4, OP>), g, dim3(mt::THREADS), mt::lds_bytes<4>(), s, p);
  } else {
    if (!moelb_allow_lds(train_rows_kernel<2, OP>, mt::lds_bytes<2>())) return MOELB_ELAUNCH;
    hipLaunchKernelGGL((train_rows_kernel<2, OP>), g, dim3(mt::THREADS), mt::lds_bytes<2>(), s, p);
  }
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

template <typename T>
int launch_sum(const TrainArgs<T>& p, int M, int N, hipStream_t s) {
  const size_t n8 = (size_t)p.E * M * N / 8;
  hipLaunchKernelGGL((sum_splits_kernel<T>), dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s, p.part, p.splits, n8,
                     p.out);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }

// Widths of the calls: a gathered row past the end plus a column stays outside
// (mt::GONE), and no tile count overflows.
constexpr int MAX_WIDTH = 1 << 19;

// What both calls require of their sizes; operands of 32-bit byte offsets.
bool sizes_ok(int rows_x, int rows, int num_groups, int E, int G, int rank, const void* gather, int gather_k, int d,
              int inter, int dtype) {
  if (rows < 0 || rows_x < 0 || num_groups < 1 || num_groups > 32768 || E < 1 || E > MOELB_MAX_E) return false;
  if (d <= 0 || d % 8 != 0 || inter <= 0 || inter % 8 != 0 || !moelb_dtype_ok(dtype)) return false;
  if (d > MAX_WIDTH || inter > MAX_WIDTH) return false;
  if (rank >= 0 && (G < 1 || rank >= G || num_groups % E != 0)) return false;
  if (gather && gather_k < 1) return false;
  if (rows > 0 && rows_x < 1) return false;
  const size_t eb = moelb_elem_bytes(dtype), most = mt::MAX_BYTES;
  return (size_t)rows_x * d * eb < most && (size_t)rows * d * eb < most && (size_t)rows * 2 * inter * eb < most &&
         (size_t)2 * inter * d * eb < most;
}

// Whether every launch of a forward (of a backward, with the gradients that are
// asked for) stays under 2^32 threads.
bool launches_ok(int rows, int E, int d, int inter, int dtype, bool backward, bool dx, bool dw13, bool dw2) {
  TrainArgs<float> p = {};  // sizes only
  p.rows = rows, p.d = d, p.inter = inter, p.E = E;
  const int BM = tile_rows(rows, E, d, inter, dtype), BN = tile_cols(rows, E, d, inter, dtype);
  const size_t most = moelb_most_blocks(dtype == MOELB_BF16 ? mt::THREADS : mt::S_THREADS);
  if (!backward) return rows_grid(p, BM, BN / 2, inter) <= most && rows_grid(p, BM, BN, d) <= most;
  const size_t grads = (dw13 ? weights_grid(p, BM, BN, 2 * inter, d) : 0) + (dw2 ? weights_grid(p, BM, BN, d, inter) : 0) +
                       (dx ? rows_grid(p, BM, BN, d) + 7 : 0);
  return rows_grid(p, BM, BN, inter) <= most && grads <= most;
}

template <typename T>
int run_forward(TrainArgs<T> p, int BM, int BN, hipStream_t s) {
  int st = launch_rows<T, OP_UP>(p, BM, BN, s);
  return st != MOELB_OK ? st : launch_rows<T, OP_DOWN>(p, BM, BN, s);
}

template <typename T>
int run_backward(TrainArgs<T> p, int BM, int BN, T* dx, T* dw13, T* dw2, float* part2, hipStream_t s) {
  if (p.rows > 0) {
    const int st = launch_rows<T, OP_DA>(p, BM, BN, s);
    if (st != MOELB_OK) return st;
  }
  GradArgs<T> g = {p, p, p, 0, 0, 0, p.rows / p.E < 2 * p.inter};
  size_t n13 = 0, n2 = 0, nx = 0;
  g.w13.out = dw13, g.w2.out = dw2, g.x.out = dx;
  g.w2.part = part2;
  if (dw13) n13 = weights_grid(g.w13, BM, BN, 2 * p.inter, p.d);
  if (dw2) n2 = weights_grid(g.w2, BM, BN, p.d, p.inter);
  if (dx && p.rows > 0) nx = (rows_grid(g.x, BM, BN, p.d) + 7) / 8 * 8;
  const size_t grid = n13 + n2 + nx;
  if (grid == 0) return MOELB_OK;
  g.n13 = (int)n13, g.n2 = (int)n2, g.nx = (int)nx;
  const dim3 gd((unsigned)grid);
  if constexpr (sizeof(T) == 4) {
    if (BN == 64)
      hipLaunchKernelGGL((train_grads_f32_kernel<64>), gd, dim3(mt::S_THREADS), 0, s, g);
    else
      hipLaunchKernelGGL((train_grads_f32_kernel<32>), gd, dim3(mt::S_THREADS), 0, s, g);
  } else if (BM == 256) {
    if (!moelb_allow_lds(train_grads_kernel<4>, mt::lds_bytes<4>())) return MOELB_ELAUNCH;
    hipLaunchKernelGGL((train_grads_kernel<4>), gd, dim3(mt::THREADS), mt::lds_bytes<4>(), s, g);
  } else {
    if (!moelb_allow_lds(train_grads_kernel<2>, mt::lds_bytes<2>())) return MOELB_ELAUNCH;
    hipLaunchKernelGGL((train_grads_kernel<2>), gd, dim3(mt::THREADS), mt::lds_bytes<2>(), s, g);
  }
  MOELB_CHECK_LAUNCH();
  if (dw13 && g.w13.splits > 1) {
    const int st = launch_sum(g.w13, 2 * p.inter, p.d, s);
    if (st != MOELB_OK) return st;
  }
  return dw2 && g.w2.splits > 1 ? launch_sum(g.w2, p.d, p.inter, s) : MOELB_OK;
}

}  // namespace

extern "C" int moelb_grouped_ffn_train(const void* x, int rows_x, int rows, const int32_t* group_off, int num_groups,
                                       int E, int G, int rank, const int32_t* gather, int gather_k, int d, int inter,
                                       int dtype, const void* w13, const void* w2, void* ws, size_t ws_bytes,
                                       float* z, void* y, void* stream) {
  if (!sizes_ok(rows_x, rows, num_groups, E, G, rank, gather, gather_k, d, inter, dtype)) return MOELB_EINVAL;
  if (!group_off || !w13 || !w2 || (rows > 0 && (!x || !y || !z))) return MOELB_EINVAL;
  if (misaligned(x) || misaligned(w13) || misaligned(w2) || misaligned(z) || misaligned(y)) return MOELB_EINVAL;
  const size_t need = sched_layout(rows, num_groups, E, inter, dtype, nullptr, nullptr);
  if (!ws || misaligned(ws) || ws_bytes < need) return MOELB_EWORKSPACE;
  if (rows == 0) return MOELB_OK;
  if (!launches_ok(rows, E, d, inter, dtype, false, false, false, false)) return MOELB_EINVAL;
  FfnSched sc;
  sched_layout(rows, num_groups, E, inter, dtype, &sc, static_cast<char*>(ws));
  sc.wpacked = 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int BM = tile_rows(rows, E, d, inter, dtype), BN = tile_cols(rows, E, d, inter, dtype);
  const int st = launch_schedule(group_off, num_groups, E, G, rank, rows, BM, gather, gather_k, rows_x, sc, s);
  if (st != MOELB_OK) return st;
  auto run = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    TrainArgs<T> p = {};
    p.x = static_cast<const T*>(x);
    p.rows_x = rows_x;
    p.w13 = static_cast<const T*>(w13);
    p.w2 = static_cast<const T*>(w2);
    p.z = z;
    p.a = static_cast<T*>(sc.amid);
    p.out = static_cast<T*>(y);
    p.rows = rows, p.d = d, p.inter = inter, p.E = E, p.s = sc;
    // 256-row tiles: the down product is moelb_grouped_ffn's, on the same
    // schedule and activations, where it streams whole K steps: it lets a tile's
    // stores run beside the next tile's loads (634 -> 520 us at 131072 rows, d =
    // 2048, inter = 1024).  With a K tail (inter = 1032) its staged form is
    // the slower one.
    if (BM == 256 && inter % mt::BK == 0 && inter >= 3 * mt::BK) {
      const int up = launch_rows<T, OP_UP>(p, BM, BN, s);
      if (up != MOELB_OK) return up;
      return moelb_grouped_ffn_stages(MOELB_FFN_DOWN, x, rows_x, rows, group_off, num_groups, E, G, rank, gather,
                                      gather_k, d, inter, dtype, w13, w2, ws, ws_bytes, y, stream);
    }
    return run_forward<T>(p, BM, BN, s);
  };
  return dtype == MOELB_BF16 ? run(static_cast<uint16_t*>(nullptr)) : run(static_cast<float*>(nullptr));
}

extern "C" size_t moelb_grouped_ffn_backward_workspace_bytes(int rows, int num_groups, int E, int d, int inter,
                                                             int dtype) {
  if (rows < 0 || num_groups < 1 || num_groups > 32768 || E < 1 || E > MOELB_MAX_E || d < 1 || d > MAX_WIDTH ||
      inter < 1 || inter > MAX_WIDTH || !moelb_dtype_ok(dtype))
    return 0;
  return back_layout(rows, num_groups, E, d, inter, dtype).total;
}

extern "C" int moelb_grouped_ffn_backward(const void* dy, const void* x, int rows_x, int rows,
                                          const int32_t* group_off, int num_groups, int E, int G, int rank,
                                          const int32_t* gather, int gather_k, int d, int inter, int dtype,
                                          const void* w13, const void* w2, const float* z, void* ws, size_t ws_bytes,
                                          void* dx, void* dw13, void* dw2, void* stream) {
  if (!sizes_ok(rows_x, rows, num_groups, E, G, rank, gather, gather_k, d, inter, dtype)) return MOELB_EINVAL;
  if (!group_off || !w13 || !w2 || (rows > 0 && (!x || !dy || !z))) return MOELB_EINVAL;
  if (misaligned(x) || misaligned(dy) || misaligned(w13) || misaligned(w2) || misaligned(z) || misaligned(dx) ||
      misaligned(dw13) || misaligned(dw2))
    return MOELB_EINVAL;
  const BackLayout l = back_layout(rows, num_groups, E, d, inter, dtype);
  if (!ws || misaligned(ws) || ws_bytes < l.total) return MOELB_EWORKSPACE;
  if (!dx && !dw13 && !dw2) return MOELB_OK;
  if (!launches_ok(rows, E, d, inter, dtype, true, dx, dw13, dw2)) return MOELB_EINVAL;
  char* base = static_cast<char*>(ws);
  FfnSched sc;
  sched_layout(rows, num_groups, E, inter, dtype, &sc, base);
  sc.wpacked = 0;
  sc.order = reinterpret_cast<int32_t*>(base + l.order);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int BM = tile_rows(rows, E, d, inter, dtype), BN = tile_cols(rows, E, d, inter, dtype);
  const int st = launch_schedule(group_off, num_groups, E, G, rank, rows, BM, gather, gather_k, rows_x, sc, s);
  if (st != MOELB_OK) return st;
  auto run = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    TrainArgs<T> p = {};
    p.x = static_cast<const T*>(x);
    p.rows_x = rows_x;
    p.w13 = static_cast<const T*>(w13);
    p.w2 = static_cast<const T*>(w2);
    p.dy = static_cast<const T*>(dy);
    p.z = const_cast<float*>(z);
    p.a = static_cast<T*>(sc.amid);
    p.dz = reinterpret_cast<T*>(base + l.dz);
    p.part = reinterpret_cast<float*>(base + l.part13);
    p.rows = rows, p.d = d, p.inter = inter, p.E = E, p.s = sc;
    return run_backward<T>(p, BM, BN, static_cast<T*>(dx), static_cast<T*>(dw13), static_cast<T*>(dw2),
                           reinterpret_cast<float*>(base + l.part2), s);
  };
  return dtype == MOELB_BF16 ? run(static_cast<uint16_t*>(nullptr)) : run(static_cast<float*>(nullptr));
}
