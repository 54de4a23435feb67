// 8-bit checkpoints of a matrix's rows and back (keep.h has the format): bound by
// memory, es bytes a value on one side and 1 + 1/32 on the other.
//
// A thread takes eight columns, four neighbouring threads a block of 32; the
// block's maximum goes between them by quad permutes.  Loads and stores are one or
// two vectors of the elements' own alignment, so rows may have any width and
// stride; a row's last, partial piece goes element by element.

#include "keep.h"
#include "train.h"

namespace moe {
namespace {

template <typename T>
using Eight = T __attribute__((ext_vector_type(8), aligned(sizeof(T))));
typedef uint32_t u32x2_1 __attribute__((ext_vector_type(2), aligned(1)));

struct Piece {
  int64_t row;
  int col, left;               // columns from col on; 0 or less: past the row's end
};
__device__ __forceinline__ bool piece_of(const CheckpointArgs &a, uint32_t per_row, Piece *p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x, row = i / per_row;
  p->row = row;
  p->col = (int)(i - row * per_row) * 8;
  p->left = a.cols - p->col;
  return row < a.rows;
}

template <typename T>
__global__ __launch_bounds__(256) void save_kernel(const CheckpointArgs a, uint32_t per_row) {
  Piece p;
  if (!piece_of(a, per_row, &p)) return;       // whole groups of four threads
  const T *src = (const T *)a.src + p.row * a.ld + p.col;
  float v[8];
  if (p.left >= 8) {
    const Eight<T> w = *(const Eight<T> *)src;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)w[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < p.left ? (float)src[j] : 0.f;
  }
  float m = keep_top(v);
  m = fmaxf(m, xor_lane<1>(m));
  m = fmaxf(m, xor_lane<2>(m));
  const int X = keep_exponent(m);
  uint32_t c[2];
  keep8(v, X, a.limit, c);
  if (p.left <= 0) return;
  uint8_t *to = a.codes + p.row * a.cols + p.col;
  if (p.left >= 8) {
    *(u32x2_1 *)to = u32x2_1{c[0], c[1]};
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < p.left) to[j] = (uint8_t)(c[j / 4] >> (8 * (j & 3)));
  }
  if (p.col % 32 == 0) a.scales[p.row * (per_row / 4) + p.col / 32] = (uint8_t)(X + 127);
}

template <typename T>
__global__ __launch_bounds__(256) void load_kernel(const CheckpointArgs a, uint32_t per_row) {
  Piece p;
  if (!piece_of(a, per_row, &p) || p.left <= 0) return;
  const uint8_t *from = a.codes + p.row * a.cols + p.col;
  const uint32_t scale = a.scales[p.row * (per_row / 4) + p.col / 32];
  T *dst = (T *)a.dst + p.row * a.ld + p.col;
  float v[8];
  if (p.left >= 8) {
    const u32x2_1 c = *(const u32x2_1 *)from;
    kept8(v, c[0], c[1], scale);
    Eight<T> w;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = (T)v[j];
    __builtin_nontemporal_store(w, (Eight<T> *)dst);
  } else {
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < p.left) c[j / 4] |= (uint32_t)from[j] << (8 * (j & 3));
    kept8(v, c[0], c[1], scale);
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < p.left) dst[j] = (T)v[j];
  }
}

uint32_t pieces_per_row(const CheckpointArgs &a) { return (uint32_t)((a.cols + 31) / 32 * 4); }

}  // namespace

int64_t checkpoint_threads(const CheckpointArgs &a) { return a.rows * pieces_per_row(a) + 256; }

hipError_t launch_checkpoint_save(const CheckpointArgs &a, hipStream_t s) {
  const uint32_t per = pieces_per_row(a);
  const dim3 grid((unsigned)((a.rows * per + 255) / 256));
  if (a.dtype == MOE_DTYPE_F32) hipLaunchKernelGGL((save_kernel<float>), grid, dim3(256), 0, s, a, per);
  else hipLaunchKernelGGL((save_kernel<bf16>), grid, dim3(256), 0, s, a, per);
  return hipGetLastError();
}

hipError_t launch_checkpoint_load(const CheckpointArgs &a, hipStream_t s) {
  const uint32_t per = pieces_per_row(a);
  const dim3 grid((unsigned)((a.rows * per + 255) / 256));
  if (a.dtype == MOE_DTYPE_F32) hipLaunchKernelGGL((load_kernel<float>), grid, dim3(256), 0, s, a, per);
  else hipLaunchKernelGGL((load_kernel<bf16>), grid, dim3(256), 0, s, a, per);
  return hipGetLastError();
}

}  // namespace moe
