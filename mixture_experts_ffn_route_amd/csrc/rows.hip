// Token rows to their experts and back, and the gradients of both:
//
//   dispatch           rows[inv[t, j]] = x[t]
//   its gradient       dx[t] = sum_j drows[inv[t, j]]
//   combine            y[t] = sum_j w[t, j] rows[inv[t, j]] + add[t]
//   its gradient       drows[inv[t, j]] = w[t, j] dy[t],  dw[t, j] = rows[inv[t, j]] . dy[t]
//
// All are bound by memory.  Working from the token's side reads (or writes) each
// token row once and each sorted row once, whatever k is, and the sums over j are
// in slot order in fp32 by one thread, so results do not depend on the launch.  A
// pair whose row is outside [0, R) takes no part.
//
// A row is cut into 16-byte pieces, one a thread.  Vectors have the alignment of an
// element, so any width is taken: the last piece of a row whose width is not a
// whole number of pieces starts early enough to end with the row (and computes some
// elements twice, alike).  Rows shorter than a piece go by elements.

#include "common.h"
#include "train.h"

namespace moe {
namespace {

template <typename T, int V>
using Vec = T __attribute__((ext_vector_type(V), aligned(sizeof(T))));

template <typename T, int V>
struct Bits {
  Vec<T, V> v;
};
template <typename T>
struct Bits<T, 1> {
  T v;
};
template <typename T, int V>
__device__ __forceinline__ void widen(float (&f)[V], const T *p) {
  if constexpr (V == 1) {
    f[0] = (float)*p;
  } else {
    const Vec<T, V> w = *(const Vec<T, V> *)p;
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)w[i];
  }
}
template <typename T, int V>
__device__ __forceinline__ void narrow(T *p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = (T)f[0];
  } else {
    Vec<T, V> w;
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = (T)f[i];
    *(Vec<T, V> *)p = w;
  }
}

// Token and first column of this thread's piece; false past the last token.
template <int V>
__device__ __forceinline__ bool place(const RowsArgs &a, uint32_t pieces, int64_t *t, int *c) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x, tok = i / pieces;
  const int at = (int)(i - tok * pieces) * V;
  *t = tok;
  *c = at < a.d - V ? at : a.d - V;
  return tok < a.T;
}

template <typename T, int V>
__global__ __launch_bounds__(256) void dispatch_kernel(const RowsArgs a, uint32_t pieces) {
  int64_t t;
  int c;
  if (!place<V>(a, pieces, &t, &c)) return;
  const auto v = *(const decltype(Bits<T, V>::v) *)((const T *)a.tokens + t * a.d + c);
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const int64_t r = a.inverse[t * a.k + j];
    if (r >= 0 && r < a.R) *(decltype(Bits<T, V>::v) *)((T *)a.out_rows + r * a.d + c) = v;
  }
}

template <typename T, int V, int K>
__global__ __launch_bounds__(256) void combine_kernel(const RowsArgs a, uint32_t pieces) {
  int64_t t;
  int c;
  if (!place<V>(a, pieces, &t, &c)) return;
  float v[K][V], w[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t r = j < a.k ? a.inverse[t * a.k + j] : -1;
    const bool on = r >= 0 && r < a.R;
    w[j] = on ? (a.weights ? a.weights[t * a.k + j] : 1.f) : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) v[j][i] = 0.f;
    if (on) widen<T, V>(v[j], (const T *)a.rows + r * a.d + c);
  }
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += w[j] * v[j][i];
  if (a.tokens) {
    float b[V];
    widen<T, V>(b, (const T *)a.tokens + t * a.d + c);
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += b[i];
  }
  narrow<T, V>((T *)a.out_tokens + t * a.d + c, sum);
}

// A workgroup takes a token; a thread every blockDim-th piece of its row.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void combine_backward_kernel(const RowsArgs a, uint32_t pieces) {
  __shared__ float red[4][K];
  const int64_t t = blockIdx.x;
  int64_t r[K];
  float w[K], dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t at = j < a.k ? a.inverse[t * a.k + j] : -1;
    r[j] = at >= 0 && at < a.R ? at : -1;
    w[j] = r[j] >= 0 && a.weights ? a.weights[t * a.k + j] : 0.f;
    dot[j] = 0.f;
  }
  for (uint32_t p = threadIdx.x; p < pieces; p += blockDim.x) {
    const int at = (int)p * V, c = at < a.d - V ? at : a.d - V;
    float g[V], v[V];
    widen<T, V>(g, (const T *)a.tokens + t * a.d + c);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (r[j] < 0) continue;
      if (a.dweights) {
        widen<T, V>(v, (const T *)a.rows + r[j] * a.d + c);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i >= at) dot[j] += v[i] * g[i];           // once each
      }
      if (a.out_rows) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = w[j] * g[i];
        narrow<T, V>((T *)a.out_rows + r[j] * a.d + c, v);
      }
    }
  }
  if (!a.dweights) return;
#pragma unroll
  for (int j = 0; j < K; ++j) dot[j] = wave_sum(dot[j]);
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int j = 0; j < K; ++j) red[wave][j] = dot[j];
  __syncthreads();
  if ((int)threadIdx.x < a.k) {
    float s = 0.f;
    for (int i = 0; i < waves; ++i) s += red[i][threadIdx.x];
    a.dweights[t * a.k + threadIdx.x] = s;
  }
}

// Pieces of a row, in vectors of V elements.
uint32_t pieces_of(int d, int V) { return (uint32_t)((d + V - 1) / V); }

int waves_a_token(uint32_t pieces) { return pieces > 192 ? 4 : (int)((pieces + 63) / 64); }

unsigned blocks_of(const RowsArgs &a, uint32_t pieces) {
  return (unsigned)((a.T * pieces + 255) / 256);
}

template <typename T, int V>
hipError_t run_dispatch(const RowsArgs &a, hipStream_t s) {
  const uint32_t n = pieces_of(a.d, V);
  hipLaunchKernelGGL((dispatch_kernel<T, V>), dim3(blocks_of(a, n)), dim3(256), 0, s, a, n);
  return hipGetLastError();
}
template <typename T, int V, int K>
hipError_t run_combine(const RowsArgs &a, bool backward, hipStream_t s) {
  const uint32_t n = pieces_of(a.d, V);
  if (backward)
    hipLaunchKernelGGL((combine_backward_kernel<T, V, K>), dim3((unsigned)a.T),
                       dim3(64 * waves_a_token(n)), 0, s, a, n);
  else
    hipLaunchKernelGGL((combine_kernel<T, V, K>), dim3(blocks_of(a, n)), dim3(256), 0, s, a, n);
  return hipGetLastError();
}
template <typename T, int V>
hipError_t run_slots(const RowsArgs &a, bool backward, hipStream_t s) {
  if (a.k <= 1) return run_combine<T, V, 1>(a, backward, s);
  if (a.k <= 2) return run_combine<T, V, 2>(a, backward, s);
  if (a.k <= 4) return run_combine<T, V, 4>(a, backward, s);
  if (a.k <= 8) return run_combine<T, V, 8>(a, backward, s);
  return run_combine<T, V, 16>(a, backward, s);
}
hipError_t run_combine_of(const RowsArgs &a, bool backward, hipStream_t s) {
  if (a.dtype == MOE_DTYPE_F32)
    return a.d >= 4 ? run_slots<float, 4>(a, backward, s) : run_slots<float, 1>(a, backward, s);
  return a.d >= 8 ? run_slots<bf16, 8>(a, backward, s) : run_slots<bf16, 1>(a, backward, s);
}

}  // namespace

int64_t rows_threads(const RowsArgs &a) {
  const int V = a.dtype == MOE_DTYPE_F32 ? 4 : 8;
  const uint32_t n = pieces_of(a.d, a.d >= V ? V : 1);
  const int64_t by_token = a.T * 64 * waves_a_token(n), flat = a.T * (int64_t)n + 256;
  return by_token > flat ? by_token : flat;
}

hipError_t launch_dispatch(const RowsArgs &a, hipStream_t s) {
  if (a.dtype == MOE_DTYPE_F32) return a.d >= 4 ? run_dispatch<float, 4>(a, s) : run_dispatch<float, 1>(a, s);
  return a.d >= 8 ? run_dispatch<bf16, 8>(a, s) : run_dispatch<bf16, 1>(a, s);
}
hipError_t launch_combine(const RowsArgs &a, hipStream_t s) { return run_combine_of(a, false, s); }
hipError_t launch_combine_backward(const RowsArgs &a, hipStream_t s) {
  return run_combine_of(a, true, s);
}

}  // namespace moe
