// The matrix-core tile of the dense products (linear.hip) and of the experts'
// products (grouped.hip).
//
// D[M, N] = A B with A and B given either "by rows" (the contraction index is the
// contiguous one) or "by columns" (it is the row index), so no operand is
// transposed in memory.
//
// A workgroup of four waves computes a (64 MI) x (64 NI) tile, each wave a
// quarter of it as MI x NI blocks of v_mfma_f32_32x32x16_bf16 (fp32 layers:
// four v_mfma_f32_32x32x2_f32 on the same bytes).  The contraction runs in
// stages of 64 bytes per row (32 bf16 or 16 fp32) through a four-slot LDS ring
// filled by asynchronous 16-byte copies; the fragments of the next step are
// read from LDS while the MFMAs of this one run.  Column operands are read
// back transposed by ds_read_b64_tr_b16 (fp32: one dword per lane).
//
// What bounds it: 256x256 tiles take 64 KB of LDS reads and 32 KB of copies per
// 1024 MFMA cycles, so LDS is busy three quarters of the time that the matrix
// cores need at best; 128 x 128 outputs a wave (256 accumulator registers) is
// the least LDS traffic per product that the registers allow.  A round of tiles
// also has a start and an epilogue in which nothing multiplies, 14 us at 256x256,
// so short rounds are slower.  bf16 TFLOP/s: 8192^3 1220, its dx 1295 and dW 1360
// (the library's product 1310 to 1570, by the power limit's clock); 4096x8192
// ->4096 1220; 4096^3 1125 (library 1330 - 1450), 4096x2048->7168 920 (1270 - 1300),
// 4096x2048->2048 755 (945).  fp32 4096^3 142, 4096x2048->7168 139 (149 and 147).
//
// Copies are buffer loads into LDS: a piece past the end of a matrix or of the
// contraction arrives as zeros without traffic, which covers every ragged
// size.
#pragma once

#include "linear_device.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// The GEMM.
struct Matrix {
  const void *p;
  int64_t ld, rows;            // as stored: rows of ld elements, cols used
  int64_t cols;
};
struct GemmOp {
  Matrix a[2], b[2], b_up;     // contraction segments added up; b_up: swiglu
  int64_t kdim[2];             // contraction length of each segment
  int segments;
  int64_t M;                   // rows of D
  int n_tiles, parts;
  int64_t m_tiles;
  // dW of swiglu: two products of the same shape in one launch, row tiles of
  // the second (a_up^T b -> y_up) after the first's
  Matrix a_up;
  void *y_up;
  int halves;                  // 1 or 2
  float *part;                 // parts > 1: [parts][halves, or 2 for swiglu][M][ldp]
  int64_t ldp;
  Epilogue e;
};

template <typename T, bool COL, int TC>
struct Operand {
  static constexpr int ES = sizeof(T);
  static constexpr int KB = 64 / ES;           // contraction elements per stage
  static constexpr int RB = TC * ES;           // column operand: bytes of an LDS row
  // 16-byte pieces of an LDS row are permuted so that a half-wave's reads take
  // distinct banks: by rows, row r's piece c sits at c ^ (r / 8 % 4) (eight
  // rows of 64 bytes cover address bits 6-8, the four pieces bits 4-5); by
  // columns, the four rows of a transposed read sit 64 bytes apart modulo 256 (rows
  // of an odd number of 128 bytes are 128 apart by themselves; of 64 columns, dense
  // products without and with it: dx of 1000 rows, 1024 -> 1024, 9.5 us and 9.5, dW 8.8 and
  // 8.4, dW of 512 rows, 2048 -> 512, 6.7 and 6.4).
  static __device__ __forceinline__ int swz(int k) {
    return ES != 2 ? 0 : TC % 128 == 0 ? (k & 3) << 2 : (k & 2) << 1;
  }

  // Byte offset, from the stage's origin, of what lane l copies to byte 16 l of
  // unit u.
  static __device__ __forceinline__ uint32_t source(int u, int lane, int64_t ld) {
    if constexpr (!COL) {
      const int r = u * 16 + (lane >> 2);
      return (uint32_t)(r * ld * ES) + ((lane & 3) ^ ((r >> 3) & 3)) * 16;
    } else {
      const int byte = u * 1024 + lane * 16;
      const int k = byte / RB;
      return (uint32_t)(k * ld * ES) + ((byte % RB / 16) ^ swz(k)) * 16;
    }
  }
  // First contraction index, within the stage, of the piece lane l copies of a
  // row operand (a wave's units have the same parity, so the same pieces).
  static __device__ __forceinline__ int first_k(int wave, int lane) {
    return ((lane & 3) ^ ((2 * wave + (lane >> 5)) & 3)) * (16 / ES);
  }
  // One lane's fragment of the 32 rows (columns of D) from `base`, step s, of
  // the stage at `lds` + `at`.  Each address is the LDS object and one offset: the
  // compiler loses track of the object over longer chains, and then lets a read
  // wait for all copies in flight (dx and dW with 128x128 tiles took up to twice
  // as long).
  static __device__ __forceinline__ u32x4 fragment(const uint8_t *lds, uint32_t at, int base, int s,
                                                   int lane) {
    if constexpr (!COL) {
      const int r = base + (lane & 31);
      const uint32_t o = at + r * 64 + ((2 * s + (lane >> 5)) ^ ((r >> 3) & 3)) * 16;
      return *(const u32x4 *)(lds + o);
    } else if constexpr (ES == 2) {
      const int col = base + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      const int k0 = 16 * s + 8 * (lane >> 5) + ((lane & 15) >> 2);
      s16x4 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = k0 + 4 * i;
        const uint32_t o = at + k * RB + ((col >> 3) ^ swz(k)) * 16 + (col & 7) * 2;
        v[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4 *)(lds + o));
      }
      const u32x2 a = __builtin_bit_cast(u32x2, v[0]), b = __builtin_bit_cast(u32x2, v[1]);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const int col = base + (lane & 31);
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t o = at + (8 * s + 4 * (lane >> 5) + j) * RB + col * 4;
        v[j] = *(const uint32_t *)(lds + o);
      }
      return v;
    }
  }
};

// acc (32 x 32, transposed: lane l holds D's row l % 32, columns 8 (e / 4) +
// 4 (l / 32) + e % 4) += a b.
template <typename T>
__device__ __forceinline__ void mma(f32x16 &acc, const u32x4 &a, const u32x4 &b) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b),
                                                  __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(b[i]), __uint_as_float(a[i]), acc,
                                                 0, 0, 0);
  }
}

// Where an operand's next stage starts: address, bytes from there to the end of
// the matrix (a copy past it reads zeros), bytes to the stage after.
struct Cursor {
  const uint8_t *p;
  int64_t left, step;
};
template <typename T, bool COL>
__device__ __forceinline__ Cursor cursor(const Matrix &m, int64_t tile0, int64_t k0) {
  constexpr int ES = sizeof(T), KB = 64 / ES;
  const int64_t at = (COL ? k0 * m.ld + tile0 : tile0 * m.ld + k0) * ES;
  return Cursor{(const uint8_t *)m.p + at, ((m.rows - 1) * m.ld + m.cols) * ES - at,
                COL ? KB * m.ld * ES : 64};
}
__device__ __forceinline__ rsrc_t cursor_rsrc(const Cursor &c) {
  const int hi = (int)(c.left >> 32);
  const uint32_t lo = (uint32_t)c.left;
  const uint32_t n = hi < 0 ? 0 : (hi > 0 || lo > kOut) ? kOut : lo;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(c.p), 0, n, 0x00027000);
}

// 16 bytes a lane from the matrix to LDS, lane l's at to + 16 l, zeros where off is
// past the end.
template <int POLICY = 0>
__device__ __forceinline__ void copy16(rsrc_t r, uint8_t *to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void *)to, 16, off, 0, 0, POLICY);
}

// The order a step's instructions are issued in: one LDS read (of DS) after
// each of the first MFMAs (of N), the copies (of VM) spread over all of them.
// The scheduler otherwise sinks the reads to their use in the next step and
// gathers the copies at the end.
template <int I, int N, int DS, int VM>
__device__ __forceinline__ void interleave() {
  if constexpr (I < N) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);           // MFMA
    constexpr int F = N * 3 / 4 > 0 ? N * 3 / 4 : 1;             // reads end three quarters through
    constexpr int d1 = DS * (I + 1) / F < DS ? DS * (I + 1) / F : DS;
    constexpr int d0 = DS * I / F < DS ? DS * I / F : DS;
    if constexpr (d1 > d0) __builtin_amdgcn_sched_group_barrier(0x100, d1 - d0, 0);
    constexpr int v = VM * (I + 1) / N - VM * I / N;
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x010, v, 0);
    interleave<I + 1, N, DS, VM>();
  }
}

}  // namespace
}  // namespace moe
