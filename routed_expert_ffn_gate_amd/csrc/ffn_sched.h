// Row schedule of the grouped FFN (forward and training): which expert and
// rows every M tile covers, from the device's group offsets.
#pragma once

#include "common.h"

namespace {

constexpr int SCHED_MIN_BM = 64;

struct FfnSched {
  int32_t* eoff;      // [E+1]   virtual row offset of each expert
  int32_t* gvb;       // [num_groups] virtual row base of each group (capped at rows)
  int32_t* mt_e;      // [max_mtiles] expert of each M tile
  int32_t* mt_v0;     // [max_mtiles] first virtual row of each M tile
  int32_t* n_mtiles;  // [1]
  int32_t* rowmap;    // [rows] physical row of each virtual row
  int32_t* asrc;      // [rows] row of x the gate/up GEMM reads for each virtual row
  void* amid;         // [rows][inter] SwiGLU activations, virtual row order
  int32_t* order;     // [E] experts by rows, most first (ties: lower id), or null: not wanted
  int wpacked;        // W13 and W2 in the packed layout (moelb_pack_weights)
};

inline size_t max_mtiles(int rows, int E) { return (size_t)(rows + SCHED_MIN_BM - 1) / SCHED_MIN_BM + E; }

inline size_t sched_layout(int rows, int num_groups, int E, int inter, int dtype, FfnSched* s, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += moelb_align256(bytes);
    return p;
  };
  const size_t mt = max_mtiles(rows, E);
  char* p_eoff = take((size_t)(E + 1) * 4);
  char* p_gvb = take((size_t)num_groups * 4);
  char* p_mte = take(mt * 4);
  char* p_mtv = take(mt * 4);
  char* p_n = take(4);
  char* p_rm = take((size_t)rows * 4);
  char* p_as = take((size_t)rows * 4);
  char* p_am = take((size_t)rows * inter * moelb_elem_bytes(dtype));
  if (s) {
    s->eoff = reinterpret_cast<int32_t*>(p_eoff);
    s->gvb = reinterpret_cast<int32_t*>(p_gvb);
    s->mt_e = reinterpret_cast<int32_t*>(p_mte);
    s->mt_v0 = reinterpret_cast<int32_t*>(p_mtv);
    s->n_mtiles = reinterpret_cast<int32_t*>(p_n);
    s->rowmap = reinterpret_cast<int32_t*>(p_rm);
    s->asrc = reinterpret_cast<int32_t*>(p_as);
    s->amid = p_am;
    s->order = nullptr;
  }
  return off;
}

// ---------------------------------------------------------------- schedule

// Experts by their rows (eoff in LDS), most first: each thread counts the
// experts before its own.
__device__ __forceinline__ void write_order(const int* eoff, int E, int32_t* order) {
  const int e = threadIdx.x;
  if (e >= E) return;
  const int n = eoff[e + 1] - eoff[e];
  int before = 0;
  for (int f = 0; f < E; ++f) {
    const int m = eoff[f + 1] - eoff[f];
    before += m > n || (m == n && f < e);
  }
  order[before] = e;
}

// Expert-major virtual row order: every selected group of expert e gets a
// contiguous range inside e's range [eoff[e], eoff[e+1]); M tiles of BM rows
// never straddle experts.  One workgroup; the group offsets are staged
// through LDS in chunks (two passes: sizes per expert, then each group's
// start), so no thread waits on a chain of global loads.  Group g covers the
// clamped rows [lo, hi), lo = clamp(group_off[g], 0, rows), hi =
// clamp(group_off[g+1], lo, rows); an unselected group counts as empty.  The
// groups of one expert get consecutive ranges in group order, so gvb over
// g = e, e+E, e+2E, ... is non-decreasing and the next group starts where
// the previous one ends (the row map relies on this).
constexpr int SCHED_CHUNK = 4096;

__global__ __launch_bounds__(256) void sched_kernel(const int32_t* __restrict__ group_off, int num_groups, int E, int G,
                                                    int rank, int rows, int BM, FfnSched s) {
  __shared__ int goff[SCHED_CHUNK + 1];
  __shared__ int eoff[MOELB_MAX_E + 1];
  __shared__ int toff[MOELB_MAX_E + 1];
  const int tid = threadIdx.x;
  const int e = tid;
  // walk the groups of expert e, chunk by chunk: add each selected group's
  // size to run, and (write) record every group's start first, capped at rows
  // (64-bit: offsets that overlap can add up past 2^31)
  auto walk = [&](bool write, long long& run) {
    for (int base = 0; base < num_groups; base += SCHED_CHUNK) {
      const int cnt = min(SCHED_CHUNK, num_groups - base);
      __syncthreads();
      for (int i = tid; i <= cnt; i += blockDim.x) goff[i] = group_off[base + i];
      __syncthreads();
      if (e < E) {
        for (int g = base + (e - base % E + E) % E; g < base + cnt; g += E) {
          const bool sel = rank < 0 || ((g / E) % G) == rank;
          const int lo = min(max(goff[g - base], 0), rows);
          const int hi = min(max(goff[g - base + 1], lo), rows);
          if (write) s.gvb[g] = (int)min(run, (long long)rows);
          if (sel) run += hi - lo;
        }
      }
    }
  };
  long long n = 0;
  walk(false, n);
  // expert offsets (clamped to rows) and M-tile offsets: two block scans
  // (Hillis-Steele over the 256 threads, one per expert)
  auto scan = [&](long long v) {  // inclusive prefix of v over threads
    __shared__ long long part[256];
    part[tid] = v;
    __syncthreads();
    for (int o = 1; o < 256; o <<= 1) {
      const long long add = tid >= o ? part[tid - o] : 0;
      __syncthreads();
      part[tid] += add;
      __syncthreads();
    }
    return part[tid];
  };
  const long long incl = scan(e < E ? n : 0);
  const int lo_row = (int)min(incl - (e < E ? n : 0), (long long)rows);
  const int hi_row = (int)min(incl, (long long)rows);
  const int ntile = e < E ? (hi_row - lo_row + BM - 1) / BM : 0;
  const long long tincl = scan(ntile);
  if (e < E) {
    eoff[e] = lo_row;
    toff[e] = (int)(tincl - ntile);
  }
  if (e == E - 1) {
    eoff[E] = hi_row;
    toff[E] = (int)tincl;
    *s.n_mtiles = (int)tincl;
  }
  __syncthreads();
  long long start = e < E ? eoff[e] : 0;
  walk(true, start);
  if (e < E) {
    s.eoff[e] = eoff[e];
    for (int i = toff[e]; i < toff[e + 1]; ++i) {
      s.mt_e[i] = e;
      s.mt_v0[i] = eoff[e] + (i - toff[e]) * BM;
    }
  }
  if (e == 0) s.eoff[E] = eoff[E];
  if (s.order) write_order(eoff, E, s.order);
}

// Inclusive prefix of v over the 256 threads of a workgroup (4 waves):
// shuffles inside each wave, then the totals of the waves below.  part4 holds
// 4 values; every thread of the workgroup must call it.
__device__ __forceinline__ long long block_incl_scan_256(long long v, long long* part4) {
  const int lane = threadIdx.x & (MOELB_WAVE - 1), w = threadIdx.x / MOELB_WAVE;
#pragma unroll
  for (int o = 1; o < MOELB_WAVE; o <<= 1) {
    const long long y = __shfl_up(v, o, MOELB_WAVE);
    if (lane >= o) v += y;
  }
  if (lane == MOELB_WAVE - 1) part4[w] = v;
  __syncthreads();
  long long add = 0;
  for (int i = 0; i < w; ++i) add += part4[i];
  __syncthreads();  // part4 is reused by the next call
  return v + add;
}

// The schedule and the row map in one launch, for up to SCHED_FUSED_GROUPS
// groups: every workgroup stages group_off in LDS and derives the expert
// offsets and the groups' virtual bases itself (the same walk as
// sched_kernel, from LDS), then maps its 256 virtual rows as rowmap_kernel
// does; workgroup 0 also writes the tables the GEMMs read (expert offsets,
// virtual bases, M tiles, one thread per tile).  The second launch and the
// single workgroup's serial tile writes were most of the schedule's time.
constexpr int SCHED_FUSED_GROUPS = 4096;

__global__ __launch_bounds__(256) void sched_rowmap_kernel(const int32_t* __restrict__ group_off, int num_groups,
                                                           int E, int G, int rank, int rows, int BM,
                                                           const int32_t* __restrict__ gather, int gather_k,
                                                           int rows_x, FfnSched s) {
  __shared__ int goff[SCHED_FUSED_GROUPS + 1];
  __shared__ int gvb[SCHED_FUSED_GROUPS];
  __shared__ int eoff[MOELB_MAX_E + 1];
  __shared__ int toff[MOELB_MAX_E + 1];
  __shared__ long long part4[4];
  const int tid = threadIdx.x;
  const int e = tid;
  for (int i = tid; i <= num_groups; i += blockDim.x) goff[i] = group_off[i];
  __syncthreads();
  // rows of expert e's selected groups (clamped as in sched_kernel)
  long long n = 0;
  if (e < E)
    for (int g = e; g < num_groups; g += E) {
      const bool sel = rank < 0 || ((g / E) % G) == rank;
      const int lo = min(max(goff[g], 0), rows);
      const int hi = min(max(goff[g + 1], lo), rows);
      if (sel) n += hi - lo;
    }
  const long long incl = block_incl_scan_256(e < E ? n : 0, part4);
  const int lo_row = (int)min(incl - (e < E ? n : 0), (long long)rows);
  const int hi_row = (int)min(incl, (long long)rows);
  const int ntile = e < E ? (hi_row - lo_row + BM - 1) / BM : 0;
  const long long tincl = block_incl_scan_256(ntile, part4);
  if (e < E) {
    eoff[e] = lo_row;
    toff[e] = (int)(tincl - ntile);
    // virtual bases of e's groups, in group order from e's first row
    long long run = lo_row;
    for (int g = e; g < num_groups; g += E) {
      const bool sel = rank < 0 || ((g / E) % G) == rank;
      const int lo = min(max(goff[g], 0), rows);
      const int hi = min(max(goff[g + 1], lo), rows);
      gvb[g] = (int)min(run, (long long)rows);
      if (sel) run += hi - lo;
    }
  }
  if (e == E - 1) {
    eoff[E] = hi_row;
    toff[E] = (int)tincl;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = tid; i <= E; i += blockDim.x) s.eoff[i] = eoff[i];
    for (int g = tid; g < num_groups; g += blockDim.x) s.gvb[g] = gvb[g];
    if (tid == 0) *s.n_mtiles = toff[E];
    // tile i belongs to the last expert with toff <= i (experts without
    // tiles share their successor's offset and are skipped that way)
    for (int i = tid; i < toff[E]; i += blockDim.x) {
      int lo = 0, hi = E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (toff[mid] <= i) lo = mid; else hi = mid - 1;
      }
      s.mt_e[i] = lo;
      s.mt_v0[i] = eoff[lo] + (i - toff[lo]) * BM;
    }
    if (s.order) write_order(eoff, E, s.order);
  }
  const int v = blockIdx.x * blockDim.x + tid;
  if (v >= eoff[E]) return;
  int lo = 0, hi = E - 1;  // eoff[0] = 0 <= v
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (eoff[mid] <= v) lo = mid; else hi = mid - 1;
  }
  const int ev = lo;
  int jl = 0, jh = (num_groups - 1 - ev) / E;  // groups ev, ev+E, ... below num_groups
  while (jl < jh) {
    const int mid = (jl + jh + 1) >> 1;
    if (gvb[ev + mid * E] <= v) jl = mid; else jh = mid - 1;
  }
  const int g = ev + jl * E;
  const long long q64 = (long long)min(max(goff[g], 0), rows) + (v - gvb[g]);
  const int q = (int)min(max(q64, 0ll), (long long)rows - 1);
  s.rowmap[v] = q;
  const int src = gather ? gather[q] / gather_k : q;
  s.asrc[v] = (src >= 0 && src < rows_x) ? src : 0;
}

// Virtual -> physical row map, and the row of x each virtual row reads
// (through the gather, when the rows come straight from the unpermuted hidden
// states).  One thread per virtual row v < eoff[E]: its expert e is the last
// one with eoff[e] <= v (offsets staged in LDS), its group the last group g
// of e with gvb[g] <= v, and its physical row clamp(group_off[g]) + (v -
// gvb[g]).  So every virtual row a GEMM tile can read is written, and with a
// row in [0, rows) (by the schedule's construction, and clamped besides),
// whatever the device offsets hold.
__global__ __launch_bounds__(256) void rowmap_kernel(const int32_t* __restrict__ group_off, int num_groups, int E,
                                                     int rows, const int32_t* __restrict__ gather, int gather_k,
                                                     int rows_x, FfnSched s) {
  __shared__ int eo[MOELB_MAX_E + 1];
  for (int i = threadIdx.x; i <= E; i += blockDim.x) eo[i] = s.eoff[i];
  __syncthreads();
  const int v = blockIdx.x * blockDim.x + threadIdx.x;
  if (v >= eo[E]) return;
  int lo = 0, hi = E - 1;  // eo[0] = 0 <= v
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (eo[mid] <= v) lo = mid; else hi = mid - 1;
  }
  const int e = lo;
  int jl = 0, jh = (num_groups - 1 - e) / E;  // groups e, e+E, ... below num_groups
  while (jl < jh) {
    const int mid = (jl + jh + 1) >> 1;
    if (s.gvb[e + mid * E] <= v) jl = mid; else jh = mid - 1;
  }
  const int g = e + jl * E;
  const long long q64 = (long long)min(max(group_off[g], 0), rows) + (v - s.gvb[g]);
  const int q = (int)min(max(q64, 0ll), (long long)rows - 1);
  s.rowmap[v] = q;
  const int src = gather ? gather[q] / gather_k : q;
  s.asrc[v] = (src >= 0 && src < rows_x) ? src : 0;
}

// XCD-aware tile id: workgroups go round-robin over 8 XCDs; give each XCD a
// contiguous range of tiles.  Returns -1 for workgroups with no tile.
__device__ __forceinline__ int xcd_tile(int bid, int total) {
  const int per = (total + 7) / 8;
  const int t = (bid & 7) * per + (bid >> 3);
  return ((bid >> 3) < per && t < total) ? t : -1;
}

// Grouped tile order: GROUP_M consecutive M tiles x every N tile, M fastest.
// The ~32 tiles an XCD runs at once then share a few A row blocks and weight
// slices, which its L2 serves, instead of streaming a whole expert's weights
// per M tile.
constexpr int GROUP_M = 8;
__device__ __forceinline__ void grouped_tile(int t, int n_mtiles, int ntn, int& mt, int& nt, int GM = GROUP_M) {
  const int group = t / (GM * ntn);
  const int first = group * GM;
  const int gm = min(GM, n_mtiles - first);
  const int local = t - group * GM * ntn;
  nt = local / gm;
  mt = first + local % gm;
}

// The schedule of one FFN call, enqueued on s.
inline int launch_schedule(const int32_t* group_off, int num_groups, int E, int G, int rank, int rows, int BM,
                           const int32_t* gather, int gather_k, int rows_x, const FfnSched& sc, hipStream_t s) {
  if (num_groups <= SCHED_FUSED_GROUPS) {
    hipLaunchKernelGGL(sched_rowmap_kernel, dim3(rows > 0 ? (rows + 255) / 256 : 1), dim3(256), 0, s, group_off,
                       num_groups, E, G < 1 ? 1 : G, rank, rows, BM, gather, gather_k, rows_x, sc);
    MOELB_CHECK_LAUNCH();
    return MOELB_OK;
  }
  hipLaunchKernelGGL(sched_kernel, dim3(1), dim3(256), 0, s, group_off, num_groups, E, G < 1 ? 1 : G, rank, rows, BM,
                     sc);
  MOELB_CHECK_LAUNCH();
  if (rows > 0)
    hipLaunchKernelGGL(rowmap_kernel, dim3((rows + 255) / 256), dim3(256), 0, s, group_off, num_groups, E, rows,
                       gather, gather_k, rows_x, sc);
  MOELB_CHECK_LAUNCH();
  return MOELB_OK;
}

}  // namespace
