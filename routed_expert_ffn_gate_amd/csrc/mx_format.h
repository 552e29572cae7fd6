// Microscaled 4-bit floating point (OCP MX): blocks of 32 e2m1 numbers with a
// shared power of two 2^X, kept as the byte X + 127.
#pragma once

#include "common.h"

namespace mx {

constexpr int BLOCK = 32;

// Bytes of a row's scales: one a block, padded so that every row starts on 16.
__host__ __device__ inline int scale_bytes(int K) { return (K / BLOCK + 15) / 16 * 16; }

// X + 127 of a block whose largest magnitude has these bits: X = floor(log2) - 2,
// at least -127 (subnormals and zeros have exponent 0 here and end there too).
// Infinities and NaN (integer order puts them last): 255, the format's NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 2^X, X = -127 a subnormal.
__device__ __forceinline__ float power(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Four values over 2^X to codes in 16 bits (HI: the upper half of `old`), for the
// scale byte X + 127.  The conversion takes the exponent of its scale operand, rounds
// to nearest even and saturates at 6, the largest number.
template <bool HI>
__device__ __forceinline__ uint32_t codes4(uint32_t old, float a, float b, float c, float d, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  old = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, s, HI ? 2 : 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, c, d, s, HI ? 3 : 1);
}

// The eight numbers in w, times f.
__device__ __forceinline__ void values8(uint32_t w, float f, float* v) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  v[0] = a.x * f, v[1] = a.y * f, v[2] = b.x * f, v[3] = b.y * f;
  v[4] = c.x * f, v[5] = c.y * f, v[6] = d.x * f, v[7] = d.y * f;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace mx
