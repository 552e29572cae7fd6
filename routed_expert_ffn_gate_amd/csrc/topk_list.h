// Descending lists of the largest keys, in registers, and their merge across the
// lanes of a token (used by the gate and by the routing rule).
#pragma once

#include "common.h"

namespace {

// Sorted (descending) insertion of key x into a register list of KL keys, one
// instruction per entry: the new entry i is the median of x, the old entry i
// and the old entry i-1 (x itself where it belongs, the entry above it
// shifted down below that, the old entry above), so every entry is computed
// from the old list, last entry first, with no chain between them.
__device__ __forceinline__ uint32_t med3_u32(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
template <int KL>
__device__ __forceinline__ void list_insert(uint32_t (&l)[KL], uint32_t x) {
#pragma unroll
  for (int i = KL - 1; i > 0; --i) l[i] = med3_u32(x, l[i], l[i - 1]);
  l[0] = x > l[0] ? x : l[0];
}

// Partner key in the merge round of lane groups of 2M (DPP, no LDS round
// trip): rounds 1 and 2 swap within quads, round 4 mirrors each half-row of 8
// lanes.  Any pairing that joins the two halves of every group of 2M lanes
// merges correctly.
template <int M>
__device__ __forceinline__ uint32_t merge_partner(uint32_t v) {
  static_assert(M == 1 || M == 2 || M == 4, "token groups of 2, 4 or 8 lanes");
  constexpr int ctrl = M == 1 ? 0xB1 : M == 2 ? 0x4E : 0x141;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, false);
}

// The partner's list is sorted: its entry j ranks no higher than place j of the
// merged list, so only the places from j on can change.
template <int M, int KL>
__device__ __forceinline__ void merge_round(uint32_t (&l)[KL]) {
  uint32_t p[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) p[i] = merge_partner<M>(l[i]);
#pragma unroll
  for (int j = 0; j < KL; ++j) {
#pragma unroll
    for (int i = KL - 1; i > j; --i) l[i] = med3_u32(p[j], l[i], l[i - 1]);
    l[j] = p[j] > l[j] ? p[j] : l[j];
  }
}

}  // namespace
