// Element-wise parts of the dense product that its kernels share.
#pragma once

#include "gemm.h"
#include "linear.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t kOut = 0x80000000u;         // an offset past every resource here

template <typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T *p, int n, bool vec) {
  if (vec && n >= 8) {
    if constexpr (sizeof(T) == 2) {
      const bf16x8 w = *(const bf16x8 *)p;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)w[j];
    } else {
      const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? (float)p[j] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8], int n, bool vec) {
  if (vec && n >= 8) {
    if constexpr (sizeof(T) == 2) {
      bf16x8 w;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = (bf16)v[j];
      *(bf16x8 *)p = w;
    } else {
      *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (T)v[j];
  }
}

// Eight elements as they are stored, zeros past n, for later.
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void fetch8(Raw8<T> &r, const T *p, int n, bool vec) {
  if (vec && n >= 8) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
      const u32x4 v = ((const u32x4 *)p)[h];
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * h + j] = v[j];
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t *q = (const uint16_t *)p;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r.w[j] = (2 * j < n ? q[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)q[2 * j + 1] << 16 : 0u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = j < n ? ((const uint32_t *)p)[j] : 0u;
  }
}
template <typename T>
__device__ __forceinline__ void widen8(float (&v)[8], const Raw8<T> &r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(T) == 2)
      v[j] = __uint_as_float(j & 1 ? r.w[j / 2] & 0xffff0000u : r.w[j / 2] << 16);
    else
      v[j] = __uint_as_float(r.w[j]);
  }
}

// fp32 layers take the accurate exponential and division; before a rounding to
// bf16 the hardware ones (relative error below 2^-20 at the arguments that
// matter) do.
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : __expf(v);
}
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  const float q = 1.f + exp_of<T>(-v);
  return sizeof(T) == 4 ? 1.f / q : __builtin_amdgcn_rcpf(q);
}

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <typename T>
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
  switch (act) {
    case MOE_ACTIVATION_RELU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] > 0.f ? v[j] : (v[j] != v[j] ? v[j] : 0.f);
      break;
    case MOE_ACTIVATION_SILU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= sigmoid<T>(v[j]);
      break;
    case MOE_ACTIVATION_GELU:
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= 0.5f * erfcf(-v[j] * 0.7071067811865476f);
      break;
    case MOE_ACTIVATION_GELU_TANH:
      // 0.5 z (1 + tanh q) = z sigmoid(2q), which keeps its relative accuracy
      // for large negative z
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] *= sigmoid<T>(2.f * kGeluA * (v[j] + kGeluB * v[j] * v[j] * v[j]));
      break;
    default: break;
  }
}

// act'(z).
template <typename T>
__device__ __forceinline__ float slope(float z, int act) {
  switch (act) {
    case MOE_ACTIVATION_RELU: return z > 0.f ? 1.f : (z != z ? z : 0.f);
    case MOE_ACTIVATION_SILU: {
      const float s = sigmoid<T>(z);
      return s * (1.f + z * (1.f - s));
    }
    case MOE_ACTIVATION_GELU:
      return 0.5f * erfcf(-z * 0.7071067811865476f) + z * 0.3989422804014327f * exp_of<T>(-0.5f * z * z);
    case MOE_ACTIVATION_GELU_TANH: {
      const float s = sigmoid<T>(2.f * kGeluA * (z + kGeluB * z * z * z));
      const float t = s * (1.f - s);           // 0 far out, where z^2 may overflow
      return t > 0.f ? s + z * t * 2.f * kGeluA * (1.f + 3.f * kGeluB * z * z) : s;
    }
    default: return 1.f;
  }
}

// The value of v in storage type T, kept on v's side of the clamp: the saved
// pre-activation decides in the backward pass whether the clamp was active,
// so rounding must not carry it across (v > L has to stay above L, v <= L at
// or below it).  One step of the type towards the right side otherwise.  The
// gate has that border at L, the up value (BOTH) at -L as well.
template <typename T, bool BOTH>
__device__ __forceinline__ float saved(float v, float L) {
  const float r = (float)(T)v;
  if (sizeof(T) == 4 || !(L > 0.f)) return r;
  const float a = BOTH ? fabsf(v) : v, b = BOTH ? fabsf(r) : r;
  if ((a > L) == (b > L) || v != v) return r;
  const uint32_t bits = __float_as_uint(r);
  return __uint_as_float(a > L ? bits + 0x10000u : bits - 0x10000u);
}

// What a thread's eight columns n .. take from the biases.
template <typename T, bool DUAL>
struct Biases {
  Raw8<T> b = {}, up = {};
  __device__ __forceinline__ void fetch(const Epilogue &e, int n) {
    if (n >= e.N) return;
    if (e.bias) fetch8<T>(b, (const T *)e.bias + n, e.N - n, e.vec != 0);
    if (DUAL && e.bias_up) fetch8<T>(up, (const T *)e.bias_up + n, e.N - n, e.vec != 0);
  }
};

// y (and z) of eight columns n .. of row m from the raw products v (and u).
// Biases and res, the residual there if there is one, are loaded ahead by the
// caller: a load here would wait its full latency for every piece (5 % longer at
// 4096x2048->7168).
template <typename T, bool DUAL>
__device__ __forceinline__ void finish8(const Epilogue &e, float (&v)[8], float (&u)[8],
                                        const Biases<T, DUAL> &bias, const float (&res)[8],
                                        int64_t m, int n) {
  const int left = e.N - n;
  const bool vec = e.vec != 0;
  float b[8];
  if (e.bias) {
    widen8<T>(b, bias.b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
  }
  if constexpr (DUAL) {
    if (e.bias_up) {
      widen8<T>(b, bias.up);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += b[j];
    }
  }
  if (e.z) {
    float k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = saved<T, false>(v[j], DUAL ? e.limit : 0.f);
    store8<T>((T *)e.z + m * e.ld_z + n, k, left, vec);
    if constexpr (DUAL) {
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = saved<T, true>(u[j], e.limit);
      store8<T>((T *)e.z_up + m * e.ld_z + n, k, left, vec);
    }
  }
  if constexpr (DUAL) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float g = v[j], w = u[j];
      if (e.limit > 0.f) {                     // NaN passes
        g = g > e.limit ? e.limit : g;
        w = w > e.limit ? e.limit : (w < -e.limit ? -e.limit : w);
      }
      v[j] = g * sigmoid<T>(g) * w;
    }
  } else {
    activate8<T>(v, e.act);
  }
  if (e.residual) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += res[j];
  }
  store8<T>((T *)e.y + m * e.ld_y + n, v, left, vec);
}

// dz (swiglu: dz and du) from dy, z (and z_up).  Clamped swiglu inputs have no
// gradient whatever dy holds, nor has a zero slope.
template <typename T, bool DUAL>
__device__ __forceinline__ void grad_of(float g, float z, float u, int act, float limit, float *dz,
                                        float *du) {
  if constexpr (DUAL) {
    bool on = true, on_up = true;
    if (limit > 0.f) {
      if (z > limit) { z = limit; on = false; }
      if (u > limit) { u = limit; on_up = false; }
      if (u < -limit) { u = -limit; on_up = false; }
    }
    const float sg = sigmoid<T>(z);
    *dz = on ? g * u * sg * (1.f + z * (1.f - sg)) : 0.f;
    *du = on_up ? g * z * sg : 0.f;
  } else {
    const float sl = slope<T>(z, act);
    *dz = sl != 0.f ? g * sl : 0.f;
  }
}

}  // namespace
}  // namespace moe
