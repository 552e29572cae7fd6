// Matrix-core tile of the training and adapter kernels: one workgroup computes
// a square tile C[m, n] = sum_k A[m, k] B[n, k] whose operands lie in memory
// either with k contiguous (a "row" operand: forward weights, activations as
// the left factor) or with k as the row index and m or n contiguous (a
// "column" operand: weights in the input gradients, where the sum runs over
// their rows; both activations in the weight gradients, where it runs over
// tokens).  No operand is transposed in memory beforehand.
//
//  * Tile 64F x 64F, F = 4 (256) or F = 2 (128); 256 threads as 2 x 2 waves,
//    wave tile 32F x 32F of v_mfma_f32_32x32x16_bf16, fp32 accumulators.
//  * K steps of 64 stream memory -> LDS with buffer_load_dwordx4 ... lds into a
//    ring of five half-stages (A or B of one step; 32 KiB each at F = 4, 16 KiB
//    at F = 2, so two F = 2 workgroups share a CU): while step t computes,
//    steps t+1 and half of t+2 are in flight.  The refills are spread over the
//    step, one instruction per F MFMAs.
//  * The loads go through a buffer descriptor: a lane that asks for an offset
//    outside it gets zeros in LDS, which is how K tails and ragged token counts
//    end inside a step without a branch.  A column operand's rows past the last
//    are past the descriptor's end by themselves; a row operand's chunks past K
//    ask for OUTSIDE.  The K step goes into the scalar offset (which the range
//    check counts), so a lane's offsets stay in registers and a load costs at
//    most one vector instruction beside it: the loop's other instructions have
//    to fit between the MFMAs of the one wave a SIMD runs at F = 4.  Rows and
//    columns of C past their end repeat a valid one and are not stored.
//  * Row operand in LDS: 64F rows of 128 B, 16-byte chunks swizzled, fragments
//    by ds_read_b128.  Column operand: 64 k rows of 128F B, 64-byte segments
//    XORed with the k row, fragments by two ds_read_b64_tr_b16 (each 16 lanes
//    read 4 k rows x 16 columns and receive them transposed: lane i column i,
//    4 consecutive k).  The XOR puts the 4 rows a read touches on different
//    banks.
//  * A column operand may be gathered: k row t reads memory row idx[t].  A wave
//    holds the indices of its 16 k rows of 32 steps in 8 registers and takes
//    them by v_readlane; no LDS and no wait inside a step.
#pragma once

#include "common.h"

namespace mt {

constexpr int BK = 64;
constexpr int SLOTS = 5;
constexpr int THREADS = 256;
// Outside every descriptor: operands are under MAX_BYTES.  GONE: the row offset
// of a gathered k row past the end; a column offset (under 1 MiB) on top of it
// stays outside.
constexpr uint32_t OUTSIDE = 0xfffffff0u, GONE = 0xffe00000u;
constexpr size_t MAX_BYTES = 0xffe00000u;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

template <int F>
constexpr int half_elems() { return 64 * F * BK; }
// the ring; the epilogue stages 128 rows x 64F fp32 in the same space
template <int F>
constexpr size_t lds_bytes() { return (size_t)SLOTS * half_elems<F>() * sizeof(uint16_t); }

__device__ __forceinline__ i32x4_t descriptor(const void* p, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  i32x4_t r;
  r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  r.y = __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xffffu));
  r.z = __builtin_amdgcn_readfirstlane((int)bytes);
  r.w = 0x00020000;
  return r;
}

// 16 bytes per lane, memory (base + voff + soff) -> LDS: lane i lands at LDS
// byte address m0 + 16 i; an offset outside the descriptor writes zeros.  M0 is
// a reserved register (the build checks that no compiler code uses it).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(uint32_t voff, i32x4_t srd, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(voff), "s"(srd),
               "s"(m0), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Row operand: k contiguous.  DMA instruction j (0 .. 2F-1) of wave w fills
// the 8 LDS rows (2F w + j) * 8 ..; lane l row l / 8 of them, slot l % 8, which
// holds chunk slot ^ swizzle(row).
template <int F>
struct RowOp {
  static constexpr bool COL = false;
  i32x4_t srd;
  uint32_t off[2 * F];
  int last;    // steps below it are whole
  bool in[2];  // this lane's chunk lies below K in step `last` (even and odd instructions)
  // row(r): memory row of LDS row r, ld: elements per memory row
  template <class Row>
  __device__ __forceinline__ void init(const void* base, uint32_t bytes, int ld, int K, Row row) {
    srd = descriptor(base, bytes);
    last = K / BK;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 2 * F; ++j) {
      const int r = (wave * 2 * F + j) * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ (((r >> 1) ^ (r << 2)) & 7);
      if (j < 2) in[j] = chunk * 8 < K - last * BK;
      off[j] = ((uint32_t)row(r) * (uint32_t)ld + (uint32_t)chunk * 8u) * 2u;
    }
  }
  __device__ __forceinline__ void begin(int) {}
  __device__ __forceinline__ void issue(int t, int j, uint32_t m0) const {
    copy16(t < last || in[j & 1] ? off[j] : OUTSIDE, srd, (uint32_t)t * (BK * 2), m0);
  }
};

// Column operand: memory row = k, columns contiguous.  DMA instruction j of
// wave w fills k rows 16 w + j R .. (R = 1024 / (128 F) rows of 128F bytes);
// a lane's 16-byte slot s of its row holds chunk s with its 64-byte segment
// (s / 4) XORed with the k row.  `bytes` are those of the K memory rows, so
// that rows past them read zeros.  With GATHER, k row t reads memory row
// idx[t] clamped to [0, rows), and `bytes` are the whole buffer's.
template <int F, bool GATHER>
struct ColOp {
  static constexpr bool COL = true;
  static constexpr int R = 8 / F;
  // distinct column offsets: the XOR takes k % (2F) of k row 16 w + j R + lane
  // part, which for F = 4 repeats every 4 instructions and for F = 2 always
  static constexpr int NC = F == 4 ? 4 : 1;
  i32x4_t srd;
  uint32_t off[GATHER ? NC : 2 * F];
  uint32_t ld2;
  int K, sub;  // sub: which of an instruction's R rows this lane loads
  const int32_t* idx;
  int rows;
  uint32_t gi[GATHER ? 8 : 1];
  // columns c0 .. of N; K memory rows from `base` (or from idx)
  __device__ __forceinline__ void init(const void* base, uint32_t bytes, int ld, int K_, int c0, int N,
                                       const int32_t* idx_ = nullptr, int rows_ = 0) {
    srd = descriptor(base, bytes);
    ld2 = (uint32_t)ld * 2u;
    K = K_;
    idx = idx_;
    rows = rows_;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int slot = lane & (8 * F - 1);
    sub = lane / (64 / R);
#pragma unroll
    for (int j = 0; j < (GATHER ? NC : 2 * F); ++j) {
      const int k = wave * 16 + j * R + sub;
      const int c = c0 + ((((slot >> 2) ^ (k & (2 * F - 1))) << 2) | (slot & 3)) * 8;
      off[j] = (uint32_t)(c < N ? c : 0) * 2u + (GATHER ? 0u : (uint32_t)k * ld2);
    }
  }
  // before the first instruction of step t: row offsets for 32 steps at a time,
  // four steps a register (lane l: step l / 16, k row l % 16 of the wave)
  __device__ __forceinline__ void begin(int t) {
    if constexpr (GATHER) {
      if ((t & 31) == 0) {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int k = (t + q * 4 + (lane >> 4)) * BK + wave * 16 + (lane & 15);
          gi[q] = k < K ? (uint32_t)min(max(idx[k], 0), rows - 1) * ld2 : GONE;
        }
      } else if ((t & 3) == 0) {
#pragma unroll
        for (int q = 0; q < 7; ++q) gi[q] = gi[q + 1];
      }
    }
  }
  __device__ __forceinline__ void issue(int t, int j, uint32_t m0) const {
    if constexpr (GATHER) {
      const int l0 = (t & 3) * 16 + j * R;
      uint32_t o = __builtin_amdgcn_readlane(gi[0], l0);
#pragma unroll
      for (int q = 1; q < R; ++q) {
        const uint32_t oq = __builtin_amdgcn_readlane(gi[0], l0 + q);
        o = sub >= q ? oq : o;
      }
      copy16(o + off[j & (NC - 1)], srd, 0, m0);
    } else {
      copy16(off[j], srd, (uint32_t)t * (BK * ld2), m0);
    }
  }
};

// LDS element offset (inside a half-stage) of this lane's fragments.
// Row operand: sub-step ks, block i = 32 rows: at[ks] + (row offset of block i) * 64.
// Column operand: at[h * F + i] + ks * 16 * 64F, h = the k half of the fragment.
template <int F, bool COL>
struct FragAt {
  int at[COL ? 2 * F : 4];
  __device__ __forceinline__ void init(int w /* wave's index along this operand */, int row0 /* row operand: its first row */) {
    const int lane = threadIdx.x & 63;
    const int fr = lane & 31, fh = lane >> 5;
    if constexpr (!COL) {
      const int sw = ((fr >> 1) ^ (fr << 2)) & 7;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) at[ks] = (row0 + fr) * BK + (((ks * 2 + fh) ^ sw) * 8);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < F; ++i) {
          const int k = fh * 8 + h * 4 + ((lane >> 2) & 3);
          const int seg = (w * F + i) ^ (k & (2 * F - 1));
          at[h * F + i] = k * 64 * F + seg * 32 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
        }
    }
  }
  __device__ __forceinline__ bf16x8_t read(const uint16_t* half, int ks, int i, int row_off) const {
    if constexpr (!COL) {
      return *reinterpret_cast<const bf16x8_t*>(half + at[ks] + row_off * BK);
    } else {
      typedef __attribute__((address_space(3))) s16x4_t lds4_t;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t*)(half + at[i] + ks * 16 * 64 * F));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t*)(half + at[F + i] + ks * 16 * 64 * F));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Column (B row in LDS) offset of block ni of wave column wn.  GU: the first
// half of the tile's B rows are gate rows, the second half the matching up
// rows, and a wave takes the same columns of both.
template <int F, bool GU>
__device__ __forceinline__ int block_col(int wn, int ni) {
  return GU ? wn * 16 * F + (ni % (F / 2)) * 32 + (ni / (F / 2)) * 32 * F : wn * 32 * F + ni * 32;
}

// The K loop: acc[mi][ni] += A block mi x B block ni over KT >= 1 steps, from
// step `turn` (< KT) on and around.  Rows a multiple of 4 KiB apart have the
// same k on the same memory channel: workgroups that all read k = 0, then k =
// 64, ... queue there, started at different steps they spread over the
// channels (a gathered operand takes its steps in order: turn = 0).
// acc holds each 32x32 block transposed (the B fragment is the MFMA's first
// operand): lane -> row lane % 32 of block mi, element j -> column (j / 4) * 8 +
// (lane / 32) * 4 + j % 4 of block ni.
template <int F, bool GU, class OA, class OB>
__device__ __forceinline__ void k_loop(uint16_t* lds, OA& oa, OB& ob, int KT, f32x16_t (&acc)[F][F], int turn = 0) {
  constexpr int HALF = half_elems<F>();
  constexpr int NI = 2 * F;  // DMA instructions per half-stage and wave
  const uint32_t lds_u32 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  FragAt<F, OA::COL> fa;
  FragAt<F, OB::COL> fb;
  fa.init(wm, wm * 32 * F);
  fb.init(wn, block_col<F, GU>(wn, 0));
#pragma unroll
  for (int mi = 0; mi < F; ++mi)
#pragma unroll
    for (int ni = 0; ni < F; ++ni)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[mi][ni][r] = 0.f;
  const int nh = 2 * KT;
  KT = __builtin_amdgcn_readfirstlane(KT);
  turn = __builtin_amdgcn_readfirstlane(turn);
  const uint32_t dst0 = lds_u32 + (uint32_t)(wave * NI * 1024);
  // DMA instruction JJ of step T's A (B: ISB) into the slot at element offset O
#define MT_ISSUE(T, ISB, O, JJ)                                     \
  {                                                                 \
    const int t_ = (T) + turn, w_ = t_ < KT ? t_ : t_ - KT;         \
    const uint32_t m_ = dst0 + (uint32_t)((O) * 2 + (JJ) * 1024);   \
    if (ISB)                                                        \
      ob.issue(w_, (JJ), m_);                                       \
    else                                                            \
      oa.issue(w_, (JJ), m_);                                       \
  }
#define MT_RA(SA, KS, I) fa.read((SA), (KS), (I), (I) * 32)
#define MT_RB(SB, KS, I) fb.read((SB), (KS), (I), block_col<F, GU>(0, I))
  bf16x8_t xa[F], xb[F], ya[F], yb[F];
  // one 16-wide k sub-step: per block row mi, read part of the next sub-step's
  // fragments (B first), run F MFMAs, issue one DMA instruction
#define MT_SUB(FA, FB, NA, NB, SA, SB, KS, RD, DO, T, ISB, O, J0)                                             \
  _Pragma("unroll") for (int mi = 0; mi < F; ++mi) {                                                          \
    if (RD) {                                                                                                 \
      if (mi < F / 2) {                                                                                       \
        NB[2 * mi] = MT_RB(SB, KS, 2 * mi);                                                                   \
        NB[2 * mi + 1] = MT_RB(SB, KS, 2 * mi + 1);                                                           \
      } else {                                                                                                \
        NA[2 * mi - F] = MT_RA(SA, KS, 2 * mi - F);                                                           \
        NA[2 * mi - F + 1] = MT_RA(SA, KS, 2 * mi - F + 1);                                                   \
      }                                                                                                       \
    }                                                                                                         \
    _Pragma("unroll") for (int ni = 0; ni < F; ++ni)                                                          \
      acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(FB[ni], FA[mi], acc[mi][ni], 0, 0, 0);            \
    if (DO) MT_ISSUE(T, ISB, O, (J0) + mi)                                                                    \
    __builtin_amdgcn_sched_barrier(0);                                                                        \
  }
  for (int j = 0; j < SLOTS && j < nh; ++j) {
    if (j & 1)
      ob.begin(j >> 1);
    else
      oa.begin(j >> 1);
#pragma unroll
    for (int jj = 0; jj < NI; ++jj) MT_ISSUE(j >> 1, j & 1, j * HALF, jj)
  }
  {
    const int after = min(SLOTS, nh) - 2;  // half-stages that may still be in flight
    if (after >= 3)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * NI) : "memory");
    else if (after == 2)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * NI) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
#pragma unroll
  for (int i = 0; i < F; ++i) {
    xa[i] = MT_RA(lds, 0, i);
    xb[i] = MT_RB(lds + HALF, 0, i);
  }
  // One K step kt.  B1: issue the second half of B_kt+1; A2: issue A_kt+2;
  // MORE: a step follows; B2: issue the first half of B_kt+2.
#define MT_STEP(KT_, B1, A2, MORE, B2)                                                                        \
  {                                                                                                           \
    const int kt_ = (KT_);                                                                                    \
    /* slots of half-stages 2 kt .. 2 kt + 4; opaque: the fragment addresses of                               \
       every slot would otherwise be held */                                                                  \
    int o0 = slot;                                                                                            \
    asm volatile("" : "+s"(o0));                                                                              \
    const int o1 = next(o0), o2 = next(o1), o3 = next(o2), o4 = next(o3);                                     \
    slot = o2;                                                                                                \
    const uint16_t* sa = lds + o0;                                                                            \
    const uint16_t* sb = lds + o1;                                                                            \
    MT_SUB(xa, xb, ya, yb, sa, sb, 1, true, B1, kt_ + 1, true, o3, F)                                         \
    if (A2) oa.begin(kt_ + 2);                                                                                \
    MT_SUB(ya, yb, xa, xb, sa, sb, 2, true, A2, kt_ + 2, false, o4, 0)                                        \
    MT_SUB(xa, xb, ya, yb, sa, sb, 3, true, A2, kt_ + 2, false, o4, F)                                        \
    if (MORE) {                                                                                               \
      /* A_kt+2 is the only half-stage issued after B_kt+1; lgkmcnt(0): this                                  \
         wave's reads of step kt are done before any wave refills its slots */                                \
      if (B2)                                                                                                 \
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(NI) : "memory");                                  \
      else                                                                                                    \
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");                                           \
      __builtin_amdgcn_s_barrier();                                                                           \
      asm volatile("" ::: "memory");                                                                          \
    }                                                                                                         \
    const uint16_t* na = lds + o2;                                                                            \
    const uint16_t* nb = lds + o3;                                                                            \
    if (B2) ob.begin(kt_ + 2);                                                                                \
    MT_SUB(ya, yb, xa, xb, na, nb, 0, MORE, B2, kt_ + 2, true, o0, 0)                                         \
  }
  auto next = [](int o) { return o == (SLOTS - 1) * HALF ? 0 : o + HALF; };
  int slot = 0;  // element offset of A_kt's slot
  if (KT >= 4) {
    MT_STEP(0, false, false, true, true)
    for (int kt = 1; kt + 2 < KT; ++kt) MT_STEP(kt, true, true, true, true)
    MT_STEP(KT - 2, true, false, true, false)
    MT_STEP(KT - 1, false, false, false, false)
  } else {
    for (int kt = 0; kt < KT; ++kt)
      MT_STEP(kt, kt >= 1 && kt + 1 < KT, kt >= 1 && kt + 2 < KT, kt + 1 < KT, kt + 2 < KT)
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#undef MT_STEP
#undef MT_SUB
#undef MT_RA
#undef MT_RB
#undef MT_ISSUE
}

// Row blocks 2 RD, 2 RD + 1 of every wave (128 rows) from the accumulators into
// LDS as fp32: staging row r, 16-byte chunk c at c ^ (r & 15), so that the
// writes (32 rows, one chunk) and the reads (one row, consecutive chunks) are
// both free of bank conflicts.  Every wave is past its K loop afterwards; the
// caller synchronises before it reads.
template <int F, bool GU, int RD>
__device__ __forceinline__ void stage(uint16_t* lds, const f32x16_t (&acc)[F][F]) {
  constexpr int B = 64 * F;
  float* st = reinterpret_cast<float*>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int fr = lane & 31, fh = lane >> 5;
  __syncthreads();
#pragma unroll
  for (int m2 = 0; m2 < 2; ++m2) {
    const int row = wm * 64 + m2 * 32 + fr;
#pragma unroll
    for (int ni = 0; ni < F; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c4 = (block_col<F, GU>(wn, ni) + q * 8 + fh * 4) / 4;
        const f32x16_t& a = acc[2 * RD + m2][ni];
        const f32x4_t v = {a[q * 4], a[q * 4 + 1], a[q * 4 + 2], a[q * 4 + 3]};
        *reinterpret_cast<f32x4_t*>(st + row * B + ((c4 ^ (row & 15)) * 4)) = v;
      }
  }
}

// After the K loop: the tile leaves the accumulators through LDS as fp32, 128
// rows at a time, and store(row, col, v) gets 8 adjacent columns of a row; with
// GU, store(row, col, gate, up) gets the matching 8 columns of both halves.
template <int F, bool GU, int RD = 0, class Store>
__device__ __forceinline__ void drain(uint16_t* lds, const f32x16_t (&acc)[F][F], Store store) {
  constexpr int B = 64 * F;
  const float* st = reinterpret_cast<const float*>(lds);
  stage<F, GU, RD>(lds, acc);
  __syncthreads();
  constexpr int W = GU ? B / 2 : B;  // columns a row gives out
  for (int c = threadIdx.x; c < 128 * (W / 8); c += THREADS) {
    const int row = c / (W / 8), col = (c % (W / 8)) * 8;
    const int tr = (row >> 6) * 32 * F + RD * 64 + (row & 63);  // row of the tile
    auto get = [&](int col_, float* v) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(st + row * B + (((col_ / 4 + h) ^ (row & 15)) * 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[h * 4 + i] = x[i];
      }
    };
    float v[8];
    get(col, v);
    if constexpr (GU) {
      float u[8];
      get(col + B / 2, u);
      store(tr, col, v, u);
    } else {
      store(tr, col, v);
    }
  }
  if constexpr (RD + 1 < F / 2) drain<F, GU, RD + 1>(lds, acc, store);
}

// Eight values to memory in the storage type (each rounded once, to nearest even).
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_pack(v[0], v[1]), bf16x2_pack(v[2], v[3]), bf16x2_pack(v[4], v[5]),
                                            bf16x2_pack(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// The gate's s = 1 / (1 + e^-g) and 1 - s.  bf16: the hardware exponential and
// reciprocal, whose error (about |g| 2^-24 relative, from the exponent's
// rounding) is far under the type's half step.  fp32: the library's exponential
// and a true quotient; for g > 0, 1 - s = e^-g s, since s itself is near 1.
template <typename T>
__device__ __forceinline__ void sigmoid_as(float g, float& s, float& c) {
  if constexpr (sizeof(T) == 4) {
    const float e = expf(-g);
    s = 1.0f / (1.0f + e);
    c = g > 0.f ? e * s : 1.0f - s;
  } else {
    s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
    c = 1.0f - s;
  }
}
template <typename T>
__device__ __forceinline__ float silu_as(float g) {
  if constexpr (sizeof(T) == 4) return g / (1.0f + expf(-g));
  return silu_f32(g);
}

// ---------------------------------------------------------------- fp32 tile
//
// The same products for fp32 storage: tile 64 x TN (TN = 64, or 32 where a call
// has few tiles), 512 threads.  A 32 x 32 block of v_mfma_f32_32x32x2_f32 is
// bound by its own 64 cycles per instruction, so the 8 waves share the tile's
// 2 TN / 32 blocks by cutting k between them: with one wave a block a step
// of one wave's chain was the time of the small calls (tiny training step 88 ->
// 64 us).  K steps (64 or 128 wide) are loaded two ahead into registers and
// written to LDS as [k][m]; partial blocks meet in LDS in a fixed order.
// a(r, k) / b(r, k) give the address of 4 consecutive floats (along k for a
// row operand, along r for a column operand) or null for zeros.
constexpr int S_BM = 64, S_THREADS = 512;

template <int TN>
struct STile {
  static constexpr int BLOCKS = 2 * TN / 32, GROUPS = 8 / BLOCKS;  // waves that share a block
  static constexpr int BK = 32 * GROUPS;                           // 64 or 128
  static constexpr int FLOATS_A = BK * (64 + 4), FLOATS_B = BK * (TN + 4);
  static constexpr int STAGE = GROUPS * 64 * TN;  // partial blocks in the epilogue
  static constexpr int X = TN / 4 - 1 < 15 ? TN / 4 - 1 : 15;  // bits of the row their chunks are XORed with
  static constexpr int FLOATS = FLOATS_A + FLOATS_B > STAGE ? FLOATS_A + FLOATS_B : STAGE;
};

template <int TN, bool CA, bool CB, class PA, class PB>
__device__ __forceinline__ void k_loop_f32(float* lds, PA pa, PB pb, int K, f32x16_t& acc) {
  using S = STile<TN>;
  constexpr int BK = S::BK;
  float* As = lds;
  float* Bs = lds + S::FLOATS_A;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int blk = wave % S::BLOCKS, kg = wave / S::BLOCKS;  // block, k group
  const int wm = blk & 1, wn = blk >> 1;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  // R rows x BK k in pieces of 4 floats, NV a thread.  Row operand: 4 k of a
  // row; LDS stride R + 1 (scalar writes).  Column operand: 4 rows of a k; LDS
  // stride R + 4.
  auto fetch = [&](auto p, auto R_, auto col_, int k0, auto& v) {
    constexpr int R = decltype(R_)::value, NV = R * BK / 4 / S_THREADS;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * S_THREADS;
      const int r = decltype(col_)::value ? c % (R / 4) * 4 : c / (BK / 4);
      const int k = k0 + (decltype(col_)::value ? c / (R / 4) : c % (BK / 4) * 4);
      const float* q = k < K ? p(r, k) : nullptr;
      v[i] = q ? *reinterpret_cast<const float4*>(q) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  auto put = [&](float* s, auto R_, auto col_, const auto& v) {
    constexpr int R = decltype(R_)::value, NV = R * BK / 4 / S_THREADS;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * S_THREADS;
      if constexpr (decltype(col_)::value) {
        *reinterpret_cast<float4*>(s + c / (R / 4) * (R + 4) + c % (R / 4) * 4) = v[i];
      } else {
        float* q = s + c % (BK / 4) * 4 * (R + 1) + c / (BK / 4);
        q[0] = v[i].x, q[R + 1] = v[i].y, q[2 * (R + 1)] = v[i].z, q[3 * (R + 1)] = v[i].w;
      }
    }
  };
  const std::integral_constant<int, 64> ra;
  const std::integral_constant<int, TN> rb;
  const std::integral_constant<bool, CA> ca;
  const std::integral_constant<bool, CB> cb;
  float4 va[2][64 * BK / 4 / S_THREADS], vb[2][TN * BK / 4 / S_THREADS];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    fetch(pa, ra, ca, s * BK, va[s]);
    fetch(pb, rb, cb, s * BK, vb[s]);
  }
  const float* ar = As + (kg * 32 + (lane >> 5)) * (CA ? 68 : 65) + wm * 32 + (lane & 31);
  const float* br = Bs + (kg * 32 + (lane >> 5)) * (TN + (CB ? 4 : 1)) + wn * 32 + (lane & 31);
  for (int k0 = 0; k0 < K; k0 += 2 * BK) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (k0 + s * BK >= K) break;
      __syncthreads();
      put(As, ra, ca, va[s]);
      put(Bs, rb, cb, vb[s]);
      __syncthreads();
      if (k0 + (s + 2) * BK < K) {
        fetch(pa, ra, ca, k0 + (s + 2) * BK, va[s]);
        fetch(pb, rb, cb, k0 + (s + 2) * BK, vb[s]);
      }
#pragma unroll
      for (int k = 0; k < 32; k += 2)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(br[k * (TN + (CB ? 4 : 1))], ar[k * (CA ? 68 : 65)], acc, 0, 0, 0);
    }
  }
}

// The partial blocks of the k groups into LDS; the caller synchronises before
// it reads.  staged_f32: columns 4 c4 .. of tile row r, the groups added in order.
template <int TN>
__device__ __forceinline__ void stage_f32(float* st, const f32x16_t& acc) {
  using S = STile<TN>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blk = wave % S::BLOCKS, kg = wave / S::BLOCKS;
  const int row = (blk & 1) * 32 + (lane & 31);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c4 = ((blk >> 1) * 32 + q * 8 + (lane >> 5) * 4) / 4;
    const f32x4_t v = {acc[q * 4], acc[q * 4 + 1], acc[q * 4 + 2], acc[q * 4 + 3]};
    *reinterpret_cast<f32x4_t*>(st + (kg * 64 + row) * TN + ((c4 ^ (row & S::X)) * 4)) = v;
  }
}
template <int TN>
__device__ __forceinline__ f32x4_t staged_f32(const float* st, int r, int c4) {
  using S = STile<TN>;
  f32x4_t x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < S::GROUPS; ++g)
    x += *reinterpret_cast<const f32x4_t*>(st + (g * 64 + r) * TN + ((c4 ^ (r & S::X)) * 4));
  return x;
}

// As drain: GU, the first half of the tile's columns are gate, the second up.
template <int TN, bool GU, class Store>
__device__ __forceinline__ void drain_f32(float* st, const f32x16_t& acc, Store store) {
  stage_f32<TN>(st, acc);
  __syncthreads();
  constexpr int W = GU ? TN / 2 : TN;
  for (int c = threadIdx.x; c < 64 * (W / 8); c += S_THREADS) {
    const int r = c / (W / 8), col = (c % (W / 8)) * 8;
    auto get = [&](int col_, float* v) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t x = staged_f32<TN>(st, r, col_ / 4 + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[h * 4 + i] = x[i];
      }
    };
    float v[8];
    get(col, v);
    if constexpr (GU) {
      float u[8];
      get(col + TN / 2, u);
      store(r, col, v, u);
    } else {
      store(r, col, v);
    }
  }
}

// Whether a product of t4 256-row or t2 128-row tiles runs faster on the former:
// one of them a compute unit against two, in whole rounds (256 units; a
// constant, so that workspace sizes do not depend on the device).  A round of
// 512 small tiles takes 0.59 of a round of 256 large ones, and its last part
// overlaps better: 4096 x 4096 weights, 3000 tokens 131 against 154 us (small),
// 4600 tokens 186 against 268, 8192 tokens 290 against 265.
inline bool large_tiles(size_t t4, size_t t2) { return (t4 + 255) / 256 * 512 * 100 <= 59 * (t2 + 77); }

}  // namespace mt
