// 8-bit checkpoints of a matrix's rows and back (keep.h has the format): bound by
// memory, es bytes a value on one side and 1 + 1/32 on the other.
//
// A thread takes 16 bytes of a row, four (bf16) or eight neighbouring ones a block of
// 32 columns; the block's maximum goes between them by lane exchanges.  Vectors have the
// elements' own alignment, so rows may have any width and stride; a row's last, partial
// piece goes element by element.

#include "keep.h"
#include "train.h"

namespace moe {
namespace {

template <typename T>
constexpr int kN = 16 / sizeof(T);             // columns of a piece
template <typename T>
using Vec = T __attribute__((ext_vector_type(kN<T>), aligned(sizeof(T))));
// The codes of a piece; clang has no vector of one.
template <typename T>
struct Codes {
  uint32_t w[kN<T> / 4];
  __device__ __forceinline__ void load(const uint8_t *p) { __builtin_memcpy(w, p, sizeof(w)); }
  __device__ __forceinline__ void store(uint8_t *p) const { __builtin_memcpy(p, w, sizeof(w)); }
};

struct Piece {
  int64_t row;
  int col, left;               // columns from col on; 0 or less: past the row's end
};
template <typename T>
__device__ __forceinline__ bool piece_of(const CheckpointArgs &a, uint32_t per_row, uint32_t i, Piece *p) {
  const uint32_t row = i / per_row;
  p->row = row;
  p->col = (int)(i - row * per_row) * kN<T>;
  p->left = a.cols - p->col;
  return row < a.rows;
}
template <typename T>
__device__ __forceinline__ int64_t scale_of(const CheckpointArgs &a, const Piece &p) {
  return p.row * ((a.cols + 31) / 32) + p.col / 32;
}

// U pieces a thread, a workgroup's width apart, all read before the first is written, so
// that the waves that fit a CU have more under way.
template <typename T, int U>
__global__ __launch_bounds__(256) void save_kernel(const CheckpointArgs a, uint32_t per_row) {
  constexpr int N = kN<T>;
  Piece p[U];
  Vec<T> w[U];
  bool on[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    on[k] = piece_of<T>(a, per_row, (blockIdx.x * U + k) * 256u + threadIdx.x, &p[k]);
    const T *src = (const T *)a.src + p[k].row * a.ld + p[k].col;
    w[k] = Vec<T>(0);
    if (on[k] && p[k].left >= N) {
      w[k] = *(const Vec<T> *)src;
    } else if (on[k]) {
#pragma unroll
      for (int j = 0; j < N - 1; ++j)
        if (j < p[k].left) w[k][j] = src[j];
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (!on[k]) return;                        // whole blocks of columns, and the rest too
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = (float)w[k][j];
    float m = keep_top(v);
    m = fmaxf(m, xor_lane<1>(m));
    m = fmaxf(m, xor_lane<2>(m));
    if (N == 4) m = fmaxf(m, xor_lane<4>(m));
    const int X = keep_exponent(m);
    Codes<T> c;
    keep<N>(v, X, a.limit, c.w);
    uint8_t *to = a.codes + p[k].row * a.cols + p[k].col;
    if (p[k].left >= N) {
      c.store(to);
    } else {
#pragma unroll
      for (int j = 0; j < N - 1; ++j)
        if (j < p[k].left) to[j] = (uint8_t)(c.w[j / 4] >> (8 * (j & 3)));
    }
    if (p[k].col % 32 == 0 && p[k].left > 0) a.scales[scale_of<T>(a, p[k])] = (uint8_t)(X + 127);
  }
}

template <typename T, int U>
__global__ __launch_bounds__(256) void load_kernel(const CheckpointArgs a, uint32_t per_row) {
  constexpr int N = kN<T>;
  Piece p[U];
  Codes<T> c[U];
  uint32_t scale[U];
  bool on[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    on[k] = piece_of<T>(a, per_row, (blockIdx.x * U + k) * 256u + threadIdx.x, &p[k]) && p[k].left > 0;
    c[k] = {};
    scale[k] = 0;
    if (!on[k]) continue;
    const uint8_t *from = a.codes + p[k].row * a.cols + p[k].col;
    scale[k] = a.scales[scale_of<T>(a, p[k])];
    if (p[k].left >= N) {
      c[k].load(from);
    } else {
#pragma unroll
      for (int j = 0; j < N - 1; ++j)
        if (j < p[k].left) c[k].w[j / 4] |= (uint32_t)from[j] << (8 * (j & 3));
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (!on[k]) continue;
    T *dst = (T *)a.dst + p[k].row * a.ld + p[k].col;
    float v[N];
    kept<N>(v, c[k].w, scale[k]);
    if (p[k].left >= N) {
      Vec<T> w;
#pragma unroll
      for (int j = 0; j < N; ++j) w[j] = (T)v[j];
      __builtin_nontemporal_store(w, (Vec<T> *)dst);
    } else {
#pragma unroll
      for (int j = 0; j < N - 1; ++j)
        if (j < p[k].left) dst[j] = (T)v[j];
    }
  }
}

uint32_t pieces_per_row(const CheckpointArgs &a) {
  return (uint32_t)((a.cols + 31) / 32 * (a.dtype == MOE_DTYPE_F32 ? 8 : 4));
}

// Pieces a thread: four where that leaves every CU sixteen workgroups.  us with one and with
// four, the same matrix again and again, so that what fits the last cache stays there:
//   1536 columns in bf16   save             load
//        16384 rows        15.1 and 19.0     8.9 and 9.7
//        21900             17.7 and 20.2    16.0 and 15.5      (from here on four)
//        65536             59.3 and 60.1    44.6 and 43.6
//       262144              234 and 221      202 and 205
//   65536 x 2048 in fp32   saved and loaded in turn 234 and 226
// so load gains little from the border on, save from where the matrix passes that cache.
template <typename T, class F1, class F4>
hipError_t run(const CheckpointArgs &a, F1 one, F4 four, hipStream_t s) {
  const uint32_t per = pieces_per_row(a);
  const int64_t n = a.rows * per;
  if (n >= (int64_t)256 * 4 * 256 * 16)
    hipLaunchKernelGGL(four, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, s, a, per);
  else
    hipLaunchKernelGGL(one, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, per);
  return hipGetLastError();
}

}  // namespace

int64_t checkpoint_threads(const CheckpointArgs &a) { return a.rows * pieces_per_row(a) + 1024; }

hipError_t launch_checkpoint_save(const CheckpointArgs &a, hipStream_t s) {
  if (a.dtype == MOE_DTYPE_F32) return run<float>(a, save_kernel<float, 1>, save_kernel<float, 4>, s);
  return run<bf16>(a, save_kernel<bf16, 1>, save_kernel<bf16, 4>, s);
}

hipError_t launch_checkpoint_load(const CheckpointArgs &a, hipStream_t s) {
  if (a.dtype == MOE_DTYPE_F32) return run<float>(a, load_kernel<float, 1>, load_kernel<float, 4>, s);
  return run<bf16>(a, load_kernel<bf16, 1>, load_kernel<bf16, 4>, s);
}

}  // namespace moe
