// 8-bit checkpoints of activations: per block of 32 consecutive columns of a row
// one E8M0 scale 2^X and E4M3 codes of v / 2^X, nearest value, ties to even.
//
// X is the least integer with amax <= 448 2^X (448: the largest E4M3 value), so no
// value saturates and each is off by at most half a step, 2^-4 of itself (down to
// 2^-6 2^X, below which steps are 2^-9 2^X).  The MXFP8 activations of the layer's
// products take floor(log2 amax) - 8, which clips values above 448 2^X: right for
// a product's operand, whose other values keep one bit more, not for a value whose
// clamp the gradient has to see.
//
// With a clamp at L > 0 no value is carried across +-L: the gradient decides by
// the kept value whether the clamp was active.  Where the nearest code lies on the
// other side, the next one towards the value's side is taken.  There is one: a
// value above L is below or at 448 2^X.
//
// NaN and infinities take the NaN code, and amax is that of the other values.
//
// The largest X is 120.  There the nearest code of values from 248 2^120 = 1.9375 2^127 on
// is 256, whose value 2^128 no float holds: they come back as infinities.
#pragma once

#include "common.h"

namespace moe {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Largest finite magnitude of N values, whatever bits they have.
template <int N>
__device__ __forceinline__ float keep_top(const float (&v)[N]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(v[j]) < __builtin_inff() ? fabsf(v[j]) : 0.f);
  return m;
}
// The same of results of arithmetic, whose NaNs are quiet ones: a maximum with one is
// the other operand, and infinities alone need the comparison.
__device__ __forceinline__ float keep_top_of_sums(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  return m == __builtin_inff() ? keep_top(v) : m;
}

// X of a block from its largest finite magnitude.
__device__ __forceinline__ int keep_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int x = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // 1.75: 448
  return amax > 0.f ? (x < -127 ? -127 : x) : 0;
}

// 2^x for x in [-127, 127].
__device__ __forceinline__ float keep_pow2(int x) {
  return __uint_as_float(x > -127 ? (uint32_t)(x + 127) << 23 : 0x400000u);
}

// Codes of N values of a block with exponent X, four to a word.
template <int N>
__device__ __forceinline__ void keep(const float (&v)[N], int X, float limit, uint32_t (&out)[N / 4]) {
  const float to = keep_pow2(-X);
  float q[N];
#pragma unroll
  for (int j = 0; j < N; ++j) q[j] = v[j] * to;              // the conversion makes NaN of infinities
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
    out[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
  }
  if (limit > 0.f) {
    const float edge = limit * to;
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
      const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)out[h], false);
      const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)out[h], true);
      const float r[4] = {a[0], a[1], b[0], b[1]};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool over = fabsf(v[4 * h + j]) > limit, is_over = fabsf(r[j]) > edge;
        // the magnitude's low bits, so a step of the code is a step of the value;
        // neither side carries out of the byte (NaN: never over and not)
        const uint32_t one = 1u << (8 * j);
        if (fabsf(q[4 * h + j]) <= 448.f) out[h] += over == is_over ? 0u : over ? one : 0u - one;
      }
    }
  }
}

// N values from their codes and the block's scale byte.
template <int N>
__device__ __forceinline__ void kept(float (&v)[N], const uint32_t (&codes)[N / 4], uint32_t scale) {
  const float unit = keep_pow2((int)scale - 127);
#pragma unroll
  for (int h = 0; h < N / 4; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[h], false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[h], true);
    v[4 * h] = a[0] * unit;
    v[4 * h + 1] = a[1] * unit;
    v[4 * h + 2] = b[0] * unit;
    v[4 * h + 3] = b[1] * unit;
  }
}

}  // namespace
}  // namespace moe
