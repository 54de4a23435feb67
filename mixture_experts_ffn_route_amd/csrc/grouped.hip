// The experts' products on rows sorted by expert, and their gradient.  For the rows
// of expert e, offsets[e] .. offsets[e + 1]:
//
//   z = x Wg^T, u = x Wu^T, h = SiLU(min(z, L)) clamp(u, -L, L), y = h Wd^T
//   dh = dy Wd, dz and du from dh and the saved z and u, h again from them
//   dWd = dy^T h, dWg = dz^T x, dWu = du^T x, dx = dz Wg + du Wu
//
// Two launches forward and four backward, all on the matrix-core tile of tile.h:
//   up      A = x by rows,   B = Wg, Wu by rows     ending: h, and z and u saved
//   down    A = h by rows,   B = Wd by rows
//   dh      A = dy by rows,  B = Wd by columns      ending: dz, du and h
//   dx      A = dz, du by rows, B = Wg, Wu by columns (two contraction segments)
//   dWd     A = dy by columns, B = h by columns     contraction over the expert's rows
//   dWg, dWu  A = dz, du by columns, B = x by columns, one launch
//
// Where an expert's rows begin is known on the device alone: every workgroup of a
// product over rows counts the row tiles of the experts before its own (a scan over
// the offsets by one wave), so nothing waits for a list; the launch has room for
// the most row tiles that `rows` rows of E experts can make, and surplus workgroups
// leave.  Offsets are clamped to [0, rows] and to ascending ones, so whatever they
// hold no access is out of range.

#include "keep.h"
#include "tile.h"
#include "train.h"

namespace moe {
namespace {

struct GroupedOp {
  GemmOp g;                    // pointers of expert 0 and row 0
  const int32_t *offsets;
  int64_t rows;
  int E;
  int row_tiles;               // products over rows: their most
  int64_t b_expert;            // bytes from one expert's B (weights) to the next's
  int64_t out_expert;          // dW: bytes from one expert's gradient to the next's
};

// Rows of an expert.
struct Span {
  int lo, n;
};
__device__ __forceinline__ Span span_of(const GroupedOp &q, int e) {
  int lo = q.offsets[e], hi = q.offsets[e + 1];
  const int most = (int)q.rows;
  lo = lo < 0 ? 0 : (lo > most ? most : lo);
  hi = hi < lo ? lo : (hi > most ? most : hi);
  return Span{lo, hi - lo};
}

struct GroupedItem {
  int e, lo, n;                // expert, its first row and rows
  int mt, nt;
};

// Work item of this workgroup in a product over rows, tiles of TM rows.  Items go
// expert by expert, an expert's column tiles one after another with its row tiles
// inside, and each XCD takes a contiguous run of them: the rows of an expert and the
// weights of a column tile are then read through one L2.
template <int TM>
__device__ __forceinline__ bool grouped_item(const GroupedOp &q, GroupedItem *out) {
  const int lane = threadIdx.x & 63;
  const int chunk = (q.E + 63) / 64;           // consecutive experts a lane
  int mine = 0;
  for (int i = 0; i < chunk; ++i) {
    const int e = lane * chunk + i;
    if (e < q.E) mine += (span_of(q, e).n + TM - 1) / TM;
  }
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off);
    if (lane >= off) upto += o;
  }
  const int nt = q.g.n_tiles;
  const int items = __builtin_amdgcn_readlane(upto, 63) * nt;
  const int per = (items + 7) / 8;
  const int slot = (int)(blockIdx.x >> 3), item = (int)(blockIdx.x & 7) * per + slot;
  if (slot >= per || item >= items) return false;
  const int src = __ffsll((unsigned long long)__ballot(upto * nt > item)) - 1;
  // the lane that holds the item's expert walks its own
  int start = (upto - mine) * nt, e = 0, lo = 0, n = 0, first = 0;
  if (lane == src) {
    for (int i = 0; i < chunk; ++i) {
      const int c = lane * chunk + i;
      if (c >= q.E) break;
      const Span s = span_of(q, c);
      const int tiles = (s.n + TM - 1) / TM * nt;
      if (item >= start && item < start + tiles) { e = c; lo = s.lo; n = s.n; first = start; }
      start += tiles;
    }
  }
  out->e = __builtin_amdgcn_readlane(e, src);
  out->lo = __builtin_amdgcn_readlane(lo, src);
  out->n = __builtin_amdgcn_readlane(n, src);
  const int local = item - __builtin_amdgcn_readlane(first, src);
  const int high = (out->n + TM - 1) / TM;
  out->nt = local / high;
  out->mt = local - out->nt * high;
  return true;
}

template <typename T>
__device__ __forceinline__ void move(Matrix &m, const GroupedItem &it) {
  m.p = (const T *)m.p + (int64_t)it.lo * m.ld;
  m.rows = it.n;
}

// ---------------------------------------------------------------------------
// Endings: rows m of the expert's, eight columns n .. .

// Rows of sums, rounded: y and dx.
template <typename T>
struct RowsOut {
  static constexpr bool plain = false;
  struct Ahead {};
  T *y;                        // row 0 of the expert
  int N;
  __device__ __forceinline__ void fetch(Ahead &, int64_t, int) const {}
  __device__ __forceinline__ void put(const Ahead &, int64_t m, int n, float (&v)[8], float (&)[8],
                                      int) const {
    store8<T>(y + m * N + n, v, N - n, true);
  }
};

// An expert's weight gradient (both of gate and up in one launch).
template <typename T>
struct WeightOut {
  static constexpr bool plain = false;
  struct Ahead {};
  T *dw, *dw_up;
  int N;
  __device__ __forceinline__ void fetch(Ahead &, int64_t, int) const {}
  __device__ __forceinline__ void put(const Ahead &, int64_t m, int n, float (&v)[8], float (&)[8],
                                      int half) const {
    store8<T>((half ? dw_up : dw) + m * N + n, v, N - n, true);
  }
};

// Eight values of z or u in 8 bits: the four neighbouring lanes hold a block (a
// tile's columns start at multiples of 32, and so does its last block's end).
__device__ __forceinline__ void keep_piece(const float (&v)[8], float limit, uint8_t *codes,
                                           uint8_t *scales, int64_t row, int n, int N) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, keep_magnitude(v[j]));
  m = fmaxf(m, xor_lane<1>(m));
  m = fmaxf(m, xor_lane<2>(m));
  const int X = keep_exponent(m);
  uint32_t c[2];
  keep8(v, X, limit, c);
  *(u32x2 *)(codes + row * N + n) = u32x2{c[0], c[1]};
  if (n % 32 == 0) scales[row * (N / 32) + n / 32] = (uint8_t)(X + 127);
}

// h, and z and u as they are saved.
template <typename T>
struct UpOut {
  static constexpr bool plain = false;
  struct Ahead {};
  T *h;                        // row 0 of all
  moe_experts_saved s;
  int64_t lo;
  int N;
  float limit;
  __device__ __forceinline__ void fetch(Ahead &, int64_t, int) const {}
  __device__ __forceinline__ void put(const Ahead &, int64_t m, int n, float (&v)[8], float (&u)[8],
                                      int) const {
    const int64_t row = lo + m;
    if (s.kind == MOE_SAVE_MXFP8) {
      keep_piece(v, limit, (uint8_t *)s.gate, s.gate_scales, row, n, N);
      keep_piece(u, limit, (uint8_t *)s.up, s.up_scales, row, n, N);
    } else if (s.kind == MOE_SAVE_FULL) {
      float k[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = saved<T, false>(v[j], limit);
      store8<T>((T *)s.gate + row * N + n, k, N - n, true);
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = saved<T, true>(u[j], limit);
      store8<T>((T *)s.up + row * N + n, k, N - n, true);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float g = v[j], w = u[j];
      if (limit > 0.f) {                       // NaN passes
        g = g > limit ? limit : g;
        w = w > limit ? limit : (w < -limit ? -limit : w);
      }
      v[j] = g * sigmoid<T>(g) * w;
    }
    store8<T>(h + row * N + n, v, N - n, true);
  }
};

// dz, du and h from dh and the saved z and u.
template <typename T>
struct SlopeOut {
  static constexpr bool plain = false;
  struct Ahead {
    Raw8<T> z, u;              // MXFP8: codes in the first two words, the scale after
  };
  T *dz, *du, *h;
  moe_experts_saved s;
  int64_t lo;
  int N;
  float limit;
  __device__ __forceinline__ void fetch(Ahead &a, int64_t m, int n) const {
    const int64_t row = lo + m;
    if (s.kind == MOE_SAVE_MXFP8) {
      const u32x2 z = *(const u32x2 *)((const uint8_t *)s.gate + row * N + n);
      const u32x2 u = *(const u32x2 *)((const uint8_t *)s.up + row * N + n);
      const int64_t at = row * (N / 32) + n / 32;
      a.z.w[0] = z[0]; a.z.w[1] = z[1]; a.z.w[2] = s.gate_scales[at];
      a.u.w[0] = u[0]; a.u.w[1] = u[1]; a.u.w[2] = s.up_scales[at];
    } else {
      fetch8<T>(a.z, (const T *)s.gate + row * N + n, N - n, true);
      fetch8<T>(a.u, (const T *)s.up + row * N + n, N - n, true);
    }
  }
  __device__ __forceinline__ void put(const Ahead &a, int64_t m, int n, float (&v)[8], float (&)[8],
                                      int) const {
    float z[8], u[8], gz[8], gu[8];
    if (s.kind == MOE_SAVE_MXFP8) {
      kept8(z, a.z.w[0], a.z.w[1], a.z.w[2]);
      kept8(u, a.u.w[0], a.u.w[1], a.u.w[2]);
    } else {
      widen8<T>(z, a.z);
      widen8<T>(u, a.u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      grad_of<T, true>(v[j], z[j], u[j], MOE_ACTIVATION_SWIGLU, limit, &gz[j], &gu[j]);
      float g = z[j], w = u[j];
      if (limit > 0.f) {
        g = g > limit ? limit : g;
        w = w > limit ? limit : (w < -limit ? -limit : w);
      }
      v[j] = g * sigmoid<T>(g) * w;
    }
    const int64_t at = (lo + m) * N + n;
    store8<T>(dz + at, gz, N - n, true);
    store8<T>(du + at, gu, N - n, true);
    store8<T>(h + at, v, N - n, true);
  }
};

// ---------------------------------------------------------------------------
// Products over rows.
template <typename T, int MI, int NI, bool BC, bool DUAL, class OUT, class ARGS>
__device__ __forceinline__ void rows_tile(const GroupedOp &q, OUT out, ARGS place) {
  GroupedItem it;
  if (!grouped_item<64 * MI>(q, &it)) return;
  GemmOp g = q.g;
  move<T>(g.a[0], it);
  move<T>(g.a[1], it);
  g.b[0].p = (const uint8_t *)g.b[0].p + it.e * q.b_expert;
  g.b[1].p = (const uint8_t *)g.b[1].p + it.e * q.b_expert;
  g.b_up.p = (const uint8_t *)g.b_up.p + it.e * q.b_expert;
  g.M = it.n;
  place(out, it);
  gemm_tile<T, MI, NI, false, BC, DUAL>(g, it.mt, it.nt, 0, out);
}

template <typename T, int MI, int NI>
__global__ __launch_bounds__(256, MI *NI >= 8 ? 1 : 2) void up_kernel(const GroupedOp q,
                                                                      const UpOut<T> o) {
  rows_tile<T, MI, NI, false, true>(q, o, [](UpOut<T> &u, const GroupedItem &it) { u.lo = it.lo; });
}
template <typename T, int MI, int NI>
__global__ __launch_bounds__(256, MI *NI >= 8 ? 1 : 2) void down_kernel(const GroupedOp q,
                                                                        const RowsOut<T> o) {
  rows_tile<T, MI, NI, false, false>(
      q, o, [](RowsOut<T> &u, const GroupedItem &it) { u.y += (int64_t)it.lo * u.N; });
}
template <typename T, int MI, int NI>
__global__ __launch_bounds__(256, MI *NI >= 8 ? 1 : 2) void dh_kernel(const GroupedOp q,
                                                                      const SlopeOut<T> o) {
  rows_tile<T, MI, NI, true, false>(q, o, [](SlopeOut<T> &u, const GroupedItem &it) { u.lo = it.lo; });
}
template <typename T, int MI, int NI>
__global__ __launch_bounds__(256, MI *NI >= 8 ? 1 : 2) void dx_kernel(const GroupedOp q,
                                                                      const RowsOut<T> o) {
  rows_tile<T, MI, NI, true, false>(
      q, o, [](RowsOut<T> &u, const GroupedItem &it) { u.y += (int64_t)it.lo * u.N; });
}

// Weight gradients: every expert has the same tiles, those of an expert without
// rows are zeros.
template <typename T, int MI, int NI>
__global__ __launch_bounds__(256, MI *NI >= 8 ? 1 : 2) void dw_kernel(const GroupedOp q,
                                                                      const WeightOut<T> o) {
  const int tiles = (int)q.g.m_tiles * q.g.n_tiles, items = tiles * q.E;
  const int per = (items + 7) / 8;
  const int slot = (int)(blockIdx.x >> 3), item = (int)(blockIdx.x & 7) * per + slot;
  if (slot >= per || item >= items) return;
  GroupedItem it;
  it.e = item / tiles;
  const int local = item - it.e * tiles;
  const int mt = local / q.g.n_tiles, nt = local - mt * q.g.n_tiles;
  const Span s = span_of(q, it.e);
  it.lo = __builtin_amdgcn_readfirstlane(s.lo);
  it.n = __builtin_amdgcn_readfirstlane(s.n);
  GemmOp g = q.g;
  move<T>(g.a[0], it);
  move<T>(g.a_up, it);
  move<T>(g.b[0], it);
  g.kdim[0] = it.n;
  WeightOut<T> out = o;
  out.dw = (T *)((uint8_t *)o.dw + it.e * q.out_expert);
  out.dw_up = (T *)((uint8_t *)o.dw_up + it.e * q.out_expert);
  gemm_tile<T, MI, NI, true, true, false>(g, mt, nt, 0, out);
}

// ---------------------------------------------------------------------------
struct Tile {
  int mi, ni;
};

// The most row tiles of `rows` rows of E experts.
int64_t most_row_tiles(int64_t rows, int E, int tm) {
  return rows / tm + (rows < E ? rows : E);
}

GroupedOp grouped_op(const ExpertsArgs &a, int N) {
  GroupedOp q = {};
  q.offsets = a.offsets;
  q.rows = a.rows;
  q.E = a.E;
  q.g.segments = 1;
  q.g.parts = 1;
  q.g.halves = 1;
  q.g.e.N = N;
  q.g.e.vec = 1;
  return q;
}

unsigned grid_of(int64_t items) { return (unsigned)(8 * ((items + 7) / 8)); }

// Workgroups of a product over rows; sets its column tiles.
unsigned rows_grid(GroupedOp &q, const Tile &t, bool dual) {
  const int to = dual ? 32 * t.ni : 64 * t.ni;
  q.g.n_tiles = (q.g.e.N + to - 1) / to;
  return grid_of(most_row_tiles(q.rows, q.E, 64 * t.mi) * q.g.n_tiles);
}

}  // namespace

ExpertsSpace experts_space(int64_t rows, int I, int dtype, bool backward) {
  const size_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
  ExpertsSpace l = {};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  l.h = take(es * rows * I);
  l.dz = take(backward ? es * rows * I : 0);
  l.du = take(backward ? es * rows * I : 0);
  l.total = off;
  return l;
}

bool experts_launchable(const ExpertsArgs &a, bool backward) {
  // the smallest tiles make the largest launch
  const int64_t wide = a.d > a.I ? a.d : a.I, cols = (wide + 31) / 32;
  const int64_t by_rows = most_row_tiles(a.rows, a.E, 64) * cols;
  const int64_t by_expert =
      backward ? 2 * (int64_t)a.E * ((a.d + 63) / 64) * ((a.I + 63) / 64) : 0;
  return (by_rows > by_expert ? by_rows : by_expert) * 256 + 2048 < (int64_t)1 << 32;
}

namespace {

template <typename T, int MI, int NI>
hipError_t run_forward(const ExpertsArgs &a, char *ws, hipStream_t s) {
  const ExpertsSpace L = experts_space(a.rows, a.I, a.dtype, false);
  constexpr int NU = NI > 1 ? NI : 2;          // two matrices share a tile
  GroupedOp q = grouped_op(a, a.I);
  q.g.a[0] = {a.x, a.d, a.rows, a.d};
  q.g.b[0] = {a.w_gate, a.d, a.I, a.d};
  q.g.b_up = {a.w_up, a.d, a.I, a.d};
  q.b_expert = (int64_t)a.I * a.d * sizeof(T);
  q.g.kdim[0] = a.d;
  const UpOut<T> up = {(T *)(ws + L.h), a.saved, 0, a.I, a.limit};
  unsigned grid = rows_grid(q, {MI, NU}, true);
  hipLaunchKernelGGL((up_kernel<T, MI, NU>), dim3(grid), dim3(256), 0, s, q, up);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  q = grouped_op(a, a.d);
  q.g.a[0] = {ws + L.h, a.I, a.rows, a.I};
  q.g.b[0] = {a.w_down, a.I, a.d, a.I};
  q.b_expert = (int64_t)a.I * a.d * sizeof(T);
  q.g.kdim[0] = a.I;
  const RowsOut<T> down = {(T *)a.y, a.d};
  grid = rows_grid(q, {MI, NI}, false);
  hipLaunchKernelGGL((down_kernel<T, MI, NI>), dim3(grid), dim3(256), 0, s, q, down);
  return hipGetLastError();
}

// A weight gradient [N, K] of every expert: columns of A (and A_up), columns of B.
template <typename T, int MI, int NI>
hipError_t run_dw(const ExpertsArgs &a, const void *A, const void *A_up, int N, const void *B, int K,
                  void *dw, void *dw_up, hipStream_t s) {
  GroupedOp q = grouped_op(a, K);
  q.g.a[0] = {A, N, a.rows, N};
  q.g.a_up = {A_up, N, a.rows, N};
  q.g.b[0] = {B, K, a.rows, K};
  q.g.M = N;
  q.g.halves = A_up ? 2 : 1;
  q.g.m_tiles = (N + 64 * MI - 1) / (64 * MI) * q.g.halves;
  q.g.n_tiles = (K + 64 * NI - 1) / (64 * NI);
  q.out_expert = (int64_t)N * K * sizeof(T);
  const WeightOut<T> o = {(T *)dw, (T *)dw_up, K};
  hipLaunchKernelGGL((dw_kernel<T, MI, NI>), dim3(grid_of(q.g.m_tiles * q.g.n_tiles * a.E)), dim3(256),
                     0, s, q, o);
  return hipGetLastError();
}

template <typename T, int MI, int NI>
hipError_t run_backward(const ExpertsArgs &a, char *ws, hipStream_t s) {
  const ExpertsSpace L = experts_space(a.rows, a.I, a.dtype, true);
  T *h = (T *)(ws + L.h), *dz = (T *)(ws + L.dz), *du = (T *)(ws + L.du);
  hipError_t err;
  if (a.rows > 0) {
    GroupedOp q = grouped_op(a, a.I);
    q.g.a[0] = {a.dy, a.d, a.rows, a.d};
    q.g.b[0] = {a.w_down, a.I, a.d, a.I};
    q.b_expert = (int64_t)a.I * a.d * sizeof(T);
    q.g.kdim[0] = a.d;
    const SlopeOut<T> o = {dz, du, h, a.saved, 0, a.I, a.limit};
    unsigned grid = rows_grid(q, {MI, NI}, false);
    hipLaunchKernelGGL((dh_kernel<T, MI, NI>), dim3(grid), dim3(256), 0, s, q, o);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  if (a.dw_down &&
      (err = run_dw<T, MI, NI>(a, a.dy, nullptr, a.d, h, a.I, a.dw_down, nullptr, s)) != hipSuccess)
    return err;
  if (a.dw_gate || a.dw_up) {
    // both in one launch, or the one that is wanted
    const bool both = a.dw_gate && a.dw_up;
    if ((err = run_dw<T, MI, NI>(a, a.dw_gate ? dz : du, both ? du : nullptr, a.I, a.x, a.d,
                                 a.dw_gate ? a.dw_gate : a.dw_up, a.dw_up, s)) != hipSuccess)
      return err;
  }
  if (a.dx && a.rows > 0) {
    GroupedOp q = grouped_op(a, a.d);
    q.g.a[0] = {dz, a.I, a.rows, a.I};
    q.g.a[1] = {du, a.I, a.rows, a.I};
    q.g.b[0] = {a.w_gate, a.d, a.I, a.d};
    q.g.b[1] = {a.w_up, a.d, a.I, a.d};
    q.b_expert = (int64_t)a.I * a.d * sizeof(T);
    q.g.kdim[0] = q.g.kdim[1] = a.I;
    q.g.segments = 2;
    const RowsOut<T> o = {(T *)a.dx, a.d};
    unsigned grid = rows_grid(q, {MI, NI}, false);
    hipLaunchKernelGGL((dx_kernel<T, MI, NI>), dim3(grid), dim3(256), 0, s, q, o);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_experts(const ExpertsArgs &a, char *ws, hipStream_t s) {
  return a.dtype == MOE_DTYPE_F32 ? run_forward<float, 1, 1>(a, ws, s)
                                  : run_forward<bf16, 1, 1>(a, ws, s);
}

hipError_t launch_experts_backward(const ExpertsArgs &a, char *ws, hipStream_t s) {
  return a.dtype == MOE_DTYPE_F32 ? run_backward<float, 1, 1>(a, ws, s)
                                  : run_backward<bf16, 1, 1>(a, ws, s);
}

}  // namespace moe
