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
// A row is cut into 16-byte pieces.  Vectors have the alignment of an
// element, so any width is taken: the last piece of a row whose width is not a
// whole number of pieces starts early enough to end with the row (and computes some
// elements twice, alike).  Rows shorter than a piece go by elements.

#include "common.h"
#include "train.h"

namespace moe {
namespace {

template <typename T, int V>
using Vec = T __attribute__((ext_vector_type(V), aligned(sizeof(T))));

// Sorted rows are read and written past the caches (nontemporal): each once, and 8192
// tokens' are larger than the L2.  4096 tokens of 8 rows of 7168 in bf16: combine 133 us,
// so 119, dispatch 104 and 93, the gradient of combine 206 and 189.
// (x, dy and what is added are not: dispatch 93, so 113.)
template <typename T, int V>
struct Piece {
  Vec<T, V> v;
  __device__ __forceinline__ void load(const T *p) { v = *(const Vec<T, V> *)p; }
  __device__ __forceinline__ void load_once(const T *p) {
    v = __builtin_nontemporal_load((const Vec<T, V> *)p);
  }
  __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
};
template <typename T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void load_once(const T *p) { v = *p; }
  __device__ __forceinline__ float operator[](int) const { return (float)v; }
};
template <typename T, int V>
__device__ __forceinline__ void narrow(T *p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = (T)f[0];
  } else {
    Vec<T, V> w;
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = (T)f[i];
    __builtin_nontemporal_store(w, (Vec<T, V> *)p);
  }
}

// Calls f(token)(first column) for this thread's pieces.  Long rows of many tokens take
// a workgroup a token, whose indices are then scalars and whose waves read the same
// rows at the same time; otherwise the pieces of all tokens stand in one line (4096 tokens
// of 88 pieces 7.5 us, by tokens 8.9; 64 tokens of 896, dispatch, 6.4 and 8.0).  By tokens and in
// line, us a call:
//   combine, 4096 tokens of 4 rows of 256 pieces 12.6 and 13.4, of 8 of 192 20.2 and 21.2
//   dispatch of the same 12.8 and 12.7, 20.5 and 19.9
//   1024 of 8 of 192: 7.2 and 7.1 (the call from Python), of 896 24.4 and 23.8
//   4096 of 8 of 896: combine 94 and 85, with an added row 97 and 90, dispatch 92 and 90
//   16384 of 6 of 640: combine 207 and 188, dispatch 192 and 189
// so combine gains to 256 pieces; of longer rows the line is the faster since a piece's
// loads are all asked for ahead.
template <int V, bool BY_TOKEN, class F>
__device__ __forceinline__ void each_piece(const RowsArgs &a, uint32_t pieces, F f) {
  auto column = [&](uint32_t p) {
    const int at = (int)p * V;
    return at < a.d - V ? at : a.d - V;
  };
  if constexpr (BY_TOKEN) {
    const auto of_token = f((int64_t)blockIdx.x);
    for (uint32_t p = threadIdx.x; p < pieces; p += 256) of_token(column(p));
  } else {
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, t = i / pieces;
    if (t < a.T) f((int64_t)t)(column(i - t * pieces));
  }
}

template <typename T, int V, bool BY_TOKEN>
__global__ __launch_bounds__(256) void dispatch_kernel(const RowsArgs a, uint32_t pieces) {
  each_piece<V, BY_TOKEN>(a, pieces, [&](int64_t t) {
    return [&a, t](int c) {
      Piece<T, V> x;
      x.load((const T *)a.tokens + t * a.d + c);
      float v[V];                              // and back: exact
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = x[i];
#pragma unroll 4
      for (int j = 0; j < a.k; ++j) {
        const int64_t r = a.inverse[t * a.k + j];
        if (r >= 0 && r < a.R) narrow<T, V>((T *)a.out_rows + r * a.d + c, v);
      }
    };
  });
}

template <int K>
struct Sources {
  int64_t row[K];              // of a token's slots; -1: none
  float w[K];
  __device__ __forceinline__ Sources(const RowsArgs &a, int64_t t) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int64_t r = j < a.k ? a.inverse[t * a.k + j] : -1;
      row[j] = r >= 0 && r < a.R ? r : -1;
      w[j] = row[j] < 0 ? 0.f : a.weights ? a.weights[t * a.k + j] : 1.f;
    }
  }
};

template <typename T, int V, int K, bool BY_TOKEN>
__global__ __launch_bounds__(256) void combine_kernel(const RowsArgs a, uint32_t pieces) {
  each_piece<V, BY_TOKEN>(a, pieces, [&](int64_t t) {
    const Sources<K> s(a, t);
    return [&a, s, t](int c) {
      Piece<T, V> v[K], add;                   // all asked for before the first is used
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (s.row[j] >= 0) v[j].load_once((const T *)a.rows + s.row[j] * a.d + c);
      if (a.tokens) add.load((const T *)a.tokens + t * a.d + c);
      float sum[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (s.row[j] >= 0)
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] += s.w[j] * v[j][i];
      if (a.tokens)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += add[i];
      narrow<T, V>((T *)a.out_tokens + t * a.d + c, sum);
    };
  });
}

// A workgroup takes a token; a thread every blockDim-th piece of its row.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void combine_backward_kernel(const RowsArgs a, uint32_t pieces) {
  __shared__ float red[4][K];
  const int64_t t = blockIdx.x;
  const Sources<K> s(a, t);
  float dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) dot[j] = 0.f;
  for (uint32_t p = threadIdx.x; p < pieces; p += blockDim.x) {
    const int at = (int)p * V, c = at < a.d - V ? at : a.d - V;
    Piece<T, V> g, v[K];
    g.load((const T *)a.tokens + t * a.d + c);
    if (a.dweights)
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (s.row[j] >= 0) v[j].load_once((const T *)a.rows + s.row[j] * a.d + c);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (s.row[j] < 0) continue;
      if (a.dweights) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i >= at) dot[j] += v[j][i] * g[i];        // once each
      }
      if (a.out_rows) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = s.w[j] * g[i];
        narrow<T, V>((T *)a.out_rows + s.row[j] * a.d + c, o);
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
    float v = 0.f;
    for (int i = 0; i < waves; ++i) v += red[i][threadIdx.x];
    a.dweights[t * a.k + threadIdx.x] = v;
  }
}

// Pieces of a row, in vectors of V elements.
uint32_t pieces_of(int d, int V) { return (uint32_t)((d + V - 1) / V); }

int waves_a_token(uint32_t pieces) { return pieces > 192 ? 4 : (int)((pieces + 63) / 64); }

bool by_token(const RowsArgs &a, uint32_t pieces) { return pieces >= 192 && a.T >= 1024; }
unsigned blocks_of(const RowsArgs &a, uint32_t pieces) {
  return (unsigned)(by_token(a, pieces) ? a.T : (a.T * pieces + 255) / 256);
}

template <typename T, int V>
hipError_t run_dispatch(const RowsArgs &a, hipStream_t s) {
  const uint32_t n = pieces_of(a.d, V);
  const dim3 grid(blocks_of(a, n));
  if (by_token(a, n)) hipLaunchKernelGGL((dispatch_kernel<T, V, true>), grid, dim3(256), 0, s, a, n);
  else hipLaunchKernelGGL((dispatch_kernel<T, V, false>), grid, dim3(256), 0, s, a, n);
  return hipGetLastError();
}
template <typename T, int V, int K>
hipError_t run_combine(const RowsArgs &a, bool backward, hipStream_t s) {
  const uint32_t n = pieces_of(a.d, V);
  const dim3 grid(blocks_of(a, n));
  if (backward)
    hipLaunchKernelGGL((combine_backward_kernel<T, V, K>), dim3((unsigned)a.T),
                       dim3(64 * waves_a_token(n)), 0, s, a, n);
  else if (by_token(a, n))
    hipLaunchKernelGGL((combine_kernel<T, V, K, true>), grid, dim3(256), 0, s, a, n);
  else
    hipLaunchKernelGGL((combine_kernel<T, V, K, false>), grid, dim3(256), 0, s, a, n);
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
  const int64_t by_token = a.T * 256, flat = a.T * (int64_t)n + 256;
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
