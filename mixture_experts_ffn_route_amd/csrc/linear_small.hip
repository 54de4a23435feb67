// The dense product where a tile of the GEMM does not fill the GPU.
//
// few_rows_kernel, up to 16 rows of x: y = act(x W^T + b) + r is a stream of W
// (2 N K FLOP per row against N K elements read), so it goes by W's bytes.  A
// workgroup takes 16 rows of W (swiglu: 8 of W and the 8 of W_up that go with
// them); its eight waves take every eighth 128-byte piece of the contraction and
// add their sums up in LDS, in order.  W is copied whole cache lines at a time
// into the wave's own part of LDS and read back in MFMA operand order (the
// operand order straight from memory, 16 rows x 64 bytes a load, reaches 5 of
// the 7 TB/s); x comes from L2 to registers.  MFMA rows are rows of W, columns
// rows of x, so a lane ends with four consecutive columns of y.  1x7168->2x2048
// swiglu bf16 (59 MB) 11.4 us, 5.2 TB/s with launch and start; 1x5120->27648 (283
// MB) 44 us, 6.4 TB/s.
//
// small_forward_kernel and small_backward_kernel, small products: time goes by
// launches and the longest chain in a workgroup, not by bytes or MFMAs.  A
// workgroup computes a 32 x 32 tile, its eight waves splitting the contraction in
// chunks of 64 (64x64 tiles whose workgroup goes through the contraction alone
// take 23 us at 203x777->1023 fp32).  Elements are read one by one, 64
// consecutive ones a load, so any width, stride and alignment does without a
// padded copy.  The backward kernel forms dz = dy act'(z) as it reads dy and z
// and computes dx, dW and db in one launch: tiles recompute dz instead of waiting
// for it.  fp32 MFMAs for both types; the products of bf16 values are exact.
// 203x777->1023 fp32 gelu 12 us; 301x256->320 fp32 silu forward 6, backward 12 us.

#include "linear_device.h"

namespace moe {
namespace {

constexpr int kWaves = 8;

// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void mma16(f32x4 &acc, const u32x4 &a, const u32x4 &b) {
  if constexpr (sizeof(T) == 2) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), acc,
                                                 0, 0, 0);
  }
}

__device__ __forceinline__ rsrc_t bytes_at(const void *p, int64_t bytes) {
  const uint32_t n = bytes <= 0 ? 0u : bytes > (int64_t)kOut ? kOut : (uint32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, n, 0x00027000);
}

template <typename T, bool DUAL>
__device__ __forceinline__ void few_rows(const SmallArgs &a) {
  constexpr int ES = sizeof(T), NS = 4, NW = DUAL ? 8 : 16, PC = NW / 8;
  // one LDS object per ring slot: a read of one does not wait for copies into another
  __shared__ __attribute__((aligned(1024))) uint8_t L0[kWaves * 2048];
  __shared__ __attribute__((aligned(1024))) uint8_t L1[kWaves * 2048];
  __shared__ __attribute__((aligned(1024))) uint8_t L2[kWaves * 2048];
  __shared__ __attribute__((aligned(1024))) uint8_t L3[kWaves * 2048];
  __shared__ __attribute__((aligned(16))) float red[kWaves][16][20];
  uint8_t *const ring[NS] = {L0, L1, L2, L3};
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * NW, N = a.e.N, M = (int)a.M;
  const int64_t kbytes = a.K * ES, ldw = a.K * ES;
  auto left = [&](int n) { return (int64_t)(N - 1 - n) * ldw + kbytes; };
  const int nu = DUAL ? n0 : n0 + 8;
  const rsrc_t rw[2] = {bytes_at((const uint8_t *)a.w + n0 * ldw, left(n0)),
                        bytes_at((const uint8_t *)(DUAL ? a.w_up : a.w) + nu * ldw,
                                 nu < N ? left(nu) : 0)};
  const rsrc_t rx = bytes_at(a.x, ((int64_t)(M - 1) * a.ld_x + a.K) * ES);

  // the eight-column piece this thread finishes, its residual on its way
  const int ft = threadIdx.x / PC, fn = n0 + (int)(threadIdx.x % PC) * 8;
  const bool finishes = threadIdx.x < 16 * PC && ft < M && fn < N;
  Raw8<T> res = {};
  Biases<T, DUAL> bias;
  if (finishes) bias.fetch(a.e, fn);
  if (finishes && a.e.residual)
    fetch8<T>(res, (const T *)a.e.residual + ft * a.e.ld_res + fn, N - fn, a.e.vec != 0);

  const int r8 = lane >> 3, piece = (lane & 7) ^ r8;           // copies
  const int t = lane & 15, g = lane >> 4;                       // operands
  const uint32_t off_w = (uint32_t)(r8 * ldw) + piece * 16;
  const uint32_t off_x = t < M ? (uint32_t)(t * a.ld_x * ES) + g * 16 : kOut;
  const int chunks = (int)((kbytes + 127) / 128);
  const int nc = (chunks + kWaves - 1) / kWaves;
  u32x4 xr[NS][2];
  auto copy = [&](int slot, int c) {
    const uint32_t at = (uint32_t)(c * kWaves + wave) * 128, kb = (uint32_t)kbytes;
    const uint32_t ow = at + piece * 16 < kb ? off_w + at : kOut;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw[u], (MOE_LDS void *)(ring[slot] + wave * 2048 + u * 1024), 16, ow, 0, 0, 0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t k = at + s * 64 + g * 16;
      xr[slot][s] = __builtin_amdgcn_raw_buffer_load_b128(rx, k < kb ? off_x + at + s * 64 : kOut,
                                                          0, 0);
    }
  };
  f32x4 acc[2] = {};
  auto step = [&](int p, int c) {
    __builtin_amdgcn_sched_barrier(0);
    copy((p + NS - 1) % NS, c + NS - 1);       // past the end: nothing is read
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(MOE_VMCNT(4 * (NS - 1)));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t o = wave * 2048 + t * 128 + ((4 * s + g) ^ (t & 7)) * 16;
      mma16<T>(acc[s], *(const u32x4 *)(ring[p] + o), xr[p][s]);
    }
  };
#pragma unroll
  for (int p = 0; p < NS - 1; ++p) copy(p, p);
  int c = 0;
  for (; c + NS <= nc; c += NS) {
#pragma unroll
    for (int p = 0; p < NS; ++p) step(p, c + p);
  }
#pragma unroll
  for (int p = 0; p < NS - 1; ++p)
    if (c + p < nc) step(p, c + p);
  __builtin_amdgcn_s_waitcnt(0);               // no copy outlives the workgroup's LDS
  *(f32x4 *)&red[wave][t][4 * g] = acc[0] + acc[1];
  __syncthreads();
  if (!finishes) return;
  float v[8] = {}, u[8] = {}, rs[8];
  const int at = DUAL ? 0 : (int)(threadIdx.x % PC) * 8;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] += red[w][ft][at + j];
      if constexpr (DUAL) u[j] += red[w][ft][8 + j];
    }
  }
  widen8<T>(rs, res);
  finish8<T, DUAL>(a.e, v, u, bias, rs, ft, fn);
}
template <typename T, bool DUAL>
__global__ __launch_bounds__(512, 4) void few_rows_kernel(const SmallArgs a) {
  few_rows<T, DUAL>(a);
}

// ---------------------------------------------------------------------------
// 32 x 32 tiles.  A wave's chunk of an operand is 32 rows (the tile's) x 64
// contraction indices, widened to fp32 in LDS rows of 68 (16-byte reads of
// eight consecutive rows then take distinct banks).
constexpr int kChunk = 64, kLd = 68, kRed = 36;

template <typename T>
__device__ __forceinline__ float widen(uint32_t b) {
  return __uint_as_float(sizeof(T) == 2 ? b << 16 : b);
}

// Lane and load j of a chunk hold (row, k).  COL: the row index is the
// contiguous one in memory.  What lies past the end of the matrix arrives as
// zero; rows past `rows` are not used, and contraction indices past the end
// (by rows, the next row's elements) are put down as zeros.
template <bool COL>
struct Chunk {
  static __device__ __forceinline__ int row(int j, int lane) { return COL ? lane & 31 : j; }
  static __device__ __forceinline__ int k(int j, int lane) {
    return COL ? 2 * j + (lane >> 5) : lane;
  }
};

// A matrix as stored: `high` rows of `wide` elements at stride ld.
struct Stored {
  const void *p;
  int64_t ld, high, wide;
};
template <typename T, bool COL>
__device__ __forceinline__ void read_chunk(uint32_t (&v)[32], const Stored &m, int64_t r0,
                                           int64_t k0, int lane) {
  constexpr int ES = sizeof(T);
  const int64_t at = COL ? k0 * m.ld + r0 : r0 * m.ld + k0;
  const rsrc_t r = bytes_at((const uint8_t *)m.p + at * ES, ((m.high - 1) * m.ld + m.wide - at) * ES);
  const int ld = (int)m.ld * ES;
  uint32_t off = COL ? (lane >> 5) * ld + (lane & 31) * ES : lane * ES;
  asm("" : "+v"(off));                         // offsets made as they are needed, not kept
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t o = off + (COL ? 2 * j : j) * ld;
    if constexpr (ES == 2) v[j] = __builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0);
    else v[j] = __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
  }
}
// Element j of a chunk into LDS; `left`: contraction indices left from the
// chunk's first.
template <bool COL>
__device__ __forceinline__ void put(float *lds, int j, float v, int64_t left, int lane) {
  const int k = Chunk<COL>::k(j, lane);
  lds[Chunk<COL>::row(j, lane) * kLd + k] = k < left ? v : 0.f;
}
template <typename T, bool COL>
__device__ __forceinline__ void put_chunk(float *lds, const uint32_t (&v)[32], int64_t left,
                                          int lane) {
#pragma unroll
  for (int j = 0; j < 32; ++j) put<COL>(lds, j, widen<T>(v[j]), left, lane);
}

// acc (transposed: lane l holds row l % 32, columns 8 (e / 4) + 4 (l / 32) +
// e % 4) += A B over a chunk; lane half h takes k = 32 h .. of each operand.
// SUM: also the sums of A's rows over the lane's k.
template <bool SUM>
__device__ __forceinline__ void multiply_chunk(f32x16 &acc, float &sum, const float *A,
                                               const float *B, int lane) {
  const int o = (lane & 31) * kLd + 32 * (lane >> 5);
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const f32x4 va = *(const f32x4 *)(A + o + 4 * s), vb = *(const f32x4 *)(B + o + 4 * s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(vb[i], va[i], acc, 0, 0, 0);
      if constexpr (SUM) sum += va[i];
    }
  }
}

__device__ __forceinline__ void put_sums(float *red, const f32x16 &acc, int lane) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *(f32x4 *)(red + (lane & 31) * kRed + 8 * e + 4 * (lane >> 5)) =
        f32x4{acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]};
}
// Eight columns of row r: the waves' sums, added in order.
__device__ __forceinline__ void take_sums(float (&v)[8], const float *red, int r, int pc) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float *q = red + w * (2 * 32 * kLd) + r * kRed + pc * 8;
    const f32x4 x = *(const f32x4 *)q, y = *(const f32x4 *)(q + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[j] += x[j]; v[4 + j] += y[j]; }
  }
}

template <typename T, bool DUAL>
__global__ __launch_bounds__(512, 2) void small_forward_kernel(const SmallArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[kWaves][2][32 * kLd];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_tiles = (a.e.N + 31) / 32;
  const int64_t mt = blockIdx.x / n_tiles;
  const int64_t m0 = mt * 32;
  const int n0 = (int)(blockIdx.x - mt * n_tiles) * 32;
  float *A = lds[wave][0], *B = lds[wave][1];
  const int ft = threadIdx.x >> 2, fc = threadIdx.x & 3;        // the piece this thread finishes
  const int64_t fm = m0 + ft;
  const int fn = n0 + fc * 8;
  const bool finishes = threadIdx.x < 128 && fm < a.M && fn < a.e.N;
  Raw8<T> res = {};
  Biases<T, DUAL> bias;
  if (finishes) bias.fetch(a.e, fn);
  if (finishes && a.e.residual)
    fetch8<T>(res, (const T *)a.e.residual + fm * a.e.ld_res + fn, a.e.N - fn, a.e.vec != 0);
  f32x16 acc = {}, acc_up = {};
  float none = 0.f;
  for (int64_t k0 = wave * kChunk; k0 < a.K; k0 += kWaves * kChunk) {
    uint32_t ra[32], rb[32], ru[32];
    read_chunk<T, false>(ra, {a.x, a.ld_x, a.M, a.K}, m0, k0, lane);
    read_chunk<T, false>(rb, {a.w, a.K, a.e.N, a.K}, n0, k0, lane);
    if constexpr (DUAL) read_chunk<T, false>(ru, {a.w_up, a.K, a.e.N, a.K}, n0, k0, lane);
    put_chunk<T, false>(A, ra, a.K - k0, lane);
    put_chunk<T, false>(B, rb, a.K - k0, lane);
    __builtin_amdgcn_wave_barrier();
    multiply_chunk<false>(acc, none, A, B, lane);
    __builtin_amdgcn_wave_barrier();
    if constexpr (DUAL) {
      put_chunk<T, false>(B, ru, a.K - k0, lane);
      __builtin_amdgcn_wave_barrier();
      multiply_chunk<false>(acc_up, none, A, B, lane);
      __builtin_amdgcn_wave_barrier();
    }
  }
  put_sums(A, acc, lane);
  if constexpr (DUAL) put_sums(B, acc_up, lane);
  __syncthreads();
  if (!finishes) return;
  float v[8], u[8], rs[8];
  take_sums(v, lds[0][0], ft, fc);
  if constexpr (DUAL) take_sums(u, lds[0][1], ft, fc);
  widen8<T>(rs, res);
  finish8<T, DUAL>(a.e, v, u, bias, rs, fm, fn);
}

// dz (or du) of a chunk, from dy, z (and z_up) read in the same order.
template <typename T, bool DUAL, bool COL>
__device__ __forceinline__ void read_dz(uint32_t (&g)[32], uint32_t (&z)[32], uint32_t (&u)[32],
                                        const SmallArgs &a, int64_t r0, int64_t k0, int lane) {
  const int64_t N = a.e.N;
  read_chunk<T, COL>(g, {a.dy, a.ld_dy, a.M, N}, r0, k0, lane);
  if (a.z) read_chunk<T, COL>(z, {a.z, N, a.M, N}, r0, k0, lane);
  if constexpr (DUAL) read_chunk<T, COL>(u, {a.z_up, N, a.M, N}, r0, k0, lane);
}
template <typename T, bool DUAL, bool COL>
__device__ __forceinline__ void put_dz(float *lds, const uint32_t (&g)[32], const uint32_t (&z)[32],
                                       const uint32_t (&u)[32], const SmallArgs &a, bool up,
                                       int64_t left, int lane) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float dz, du = 0.f;
    grad_of<T, DUAL>(widen<T>(g[j]), a.z ? widen<T>(z[j]) : 0.f, DUAL ? widen<T>(u[j]) : 0.f,
                     a.e.act, a.e.limit, &dz, &du);
    put<COL>(lds, j, DUAL && up ? du : dz, left, lane);
  }
}

// Workgroups: dx tiles [rows / 32][in / 32], then tiles of dW (swiglu: dW, then
// dW_up) [out / 32][in / 32]; those with in-tile 0 also sum db.  Where only db is
// wanted there is that tile alone.
template <typename T, bool DUAL>
__global__ __launch_bounds__(512, 2) void small_backward_kernel(const SmallArgs a) {
  __shared__ __attribute__((aligned(16))) float lds[kWaves][2][32 * kLd];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *A = lds[wave][0], *B = lds[wave][1];
  const int64_t K = a.K, N = a.e.N;
  f32x16 acc = {};
  float sum = 0.f, none = 0.f;
  uint32_t g[32], z[32] = {}, u[32] = {}, rb[32] = {};
  int64_t item = blockIdx.x, r0, rows;
  int64_t c0;
  T *out;
  int64_t ldo;
  bool sums = false, up = false;
  if (item < a.dx_tiles) {
    const int64_t kt = (K + 31) / 32;
    r0 = item / kt * 32;
    c0 = item % kt * 32;
    rows = a.M; out = (T *)a.dx; ldo = a.ld_dx;
    const int64_t per = (N + kChunk - 1) / kChunk, all = DUAL ? 2 * per : per;
    for (int64_t c = wave; c < all; c += kWaves) {
      const bool second = DUAL && c >= per;
      const int64_t k0 = (second ? c - per : c) * kChunk;
      read_chunk<T, true>(rb, {second ? a.w_up : a.w, K, N, K}, c0, k0, lane);
      read_dz<T, DUAL, false>(g, z, u, a, r0, k0, lane);
      put_chunk<T, true>(B, rb, N - k0, lane);
      put_dz<T, DUAL, false>(A, g, z, u, a, second, N - k0, lane);
      __builtin_amdgcn_wave_barrier();
      multiply_chunk<false>(acc, none, A, B, lane);
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    item -= a.dx_tiles;
    const bool want = a.dw || a.dw_up;
    const int64_t kt = want ? (K + 31) / 32 : 1, per = (N + 31) / 32 * kt;
    up = DUAL && item >= per;
    if (up) item -= per;
    r0 = item / kt * 32;
    c0 = item % kt * 32;
    rows = N; out = (T *)(up ? a.dw_up : a.dw); ldo = K;
    void *db = up ? a.db_up : a.db;
    sums = c0 == 0 && db;
    if (!out && !sums) return;                 // uniform in the workgroup
    for (int64_t k0 = wave * kChunk; k0 < a.M; k0 += kWaves * kChunk) {
      // db alone: any finite B will do
      if (out) read_chunk<T, true>(rb, {a.x, a.ld_x, a.M, K}, c0, k0, lane);
      read_dz<T, DUAL, true>(g, z, u, a, r0, k0, lane);
      put_chunk<T, true>(B, rb, out ? a.M - k0 : 0, lane);
      put_dz<T, DUAL, true>(A, g, z, u, a, up, a.M - k0, lane);
      __builtin_amdgcn_wave_barrier();
      multiply_chunk<true>(acc, sum, A, B, lane);
      __builtin_amdgcn_wave_barrier();
    }
  }
  put_sums(A, acc, lane);
  if (sums) B[lane] = sum;
  __syncthreads();
  const int ft = threadIdx.x >> 2, fc = threadIdx.x & 3;
  if (threadIdx.x < 128 && out && r0 + ft < rows && c0 + fc * 8 < K) {
    float o[8];
    take_sums(o, lds[0][0], ft, fc);
    store8<T>(out + (r0 + ft) * ldo + c0 + fc * 8, o, (int)(K - c0 - fc * 8), false);
  }
  if (sums && threadIdx.x < 32 && r0 + threadIdx.x < N) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += lds[w][1][threadIdx.x] + lds[w][1][threadIdx.x + 32];
    ((T *)(up ? a.db_up : a.db))[r0 + threadIdx.x] = (T)s;
  }
}

}  // namespace

template <typename T>
hipError_t launch_few_rows(const SmallArgs &a, bool dual, hipStream_t s) {
  const int per = dual ? 8 : 16;
  const dim3 grid((unsigned)((a.e.N + per - 1) / per));
  if (dual) hipLaunchKernelGGL((few_rows_kernel<T, true>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((few_rows_kernel<T, false>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_small_forward(const SmallArgs &a, bool dual, hipStream_t s) {
  const dim3 grid((unsigned)((a.M + 31) / 32 * ((a.e.N + 31) / 32)));
  if (dual) hipLaunchKernelGGL((small_forward_kernel<T, true>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((small_forward_kernel<T, false>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_small_backward(SmallArgs a, bool dual, hipStream_t s) {
  const int64_t kt = (a.K + 31) / 32, nt = (a.e.N + 31) / 32;
  a.dx_tiles = a.dx ? (a.M + 31) / 32 * kt : 0;
  const bool dw = a.dw || a.dw_up, db = a.db || a.db_up;
  const int64_t rest = (dual ? 2 : 1) * nt * (dw ? kt : db ? 1 : 0);
  const dim3 grid((unsigned)(a.dx_tiles + rest));
  if (dual) hipLaunchKernelGGL((small_backward_kernel<T, true>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((small_backward_kernel<T, false>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

template hipError_t launch_few_rows<float>(const SmallArgs &, bool, hipStream_t);
template hipError_t launch_few_rows<bf16>(const SmallArgs &, bool, hipStream_t);
template hipError_t launch_small_forward<float>(const SmallArgs &, bool, hipStream_t);
template hipError_t launch_small_forward<bf16>(const SmallArgs &, bool, hipStream_t);
template hipError_t launch_small_backward<float>(SmallArgs, bool, hipStream_t);
template hipError_t launch_small_backward<bf16>(SmallArgs, bool, hipStream_t);

}  // namespace moe
