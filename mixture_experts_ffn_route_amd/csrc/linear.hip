// Dense product with bias, activation and residual, and its gradient:
//
//   z = x W^T + b,  y = act(z) + r                 (swiglu: two products)
//   dz = dy act'(z), dx = dz W, dW = dz^T x, db = sum over rows of dz
//
// One GEMM tile (tile.h) serves the three products, so no operand is transposed in
// memory:
//   forward  A = x  by rows,        B = W  by rows
//   dx       A = dz by rows,        B = W  by columns (contraction over out)
//   dW       A = dz by columns,     B = x  by columns (contraction over rows)
// Rows that are not whole 16-byte pieces (odd widths or strides) are
// first copied to padded rows in the workspace.

#include "tile.h"

namespace moe {
namespace {

// Work item of this workgroup: workgroups are dealt round-robin to the 8 XCDs,
// each XCD takes a contiguous run of items; within a part, tiles run down
// groups of 8 row tiles before the next column tile, so the tiles an XCD works
// on at a time form a block that shares operand rows in its L2.
__device__ __forceinline__ bool gemm_item(const GemmOp &g, int64_t *mt, int *nt, int *part) {
  const int64_t tiles = g.m_tiles * g.n_tiles, items = tiles * g.parts;
  const int64_t per = (items + 7) / 8;
  const int64_t item = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || item >= items) return false;
  *part = (int)(item / tiles);
  const int64_t t = item - *part * tiles;
  const int64_t group = t / (8 * g.n_tiles), first = group * 8;
  const int64_t high = g.m_tiles - first < 8 ? g.m_tiles - first : 8;
  const int64_t r = t - first * g.n_tiles;
  *nt = (int)(r / high);
  *mt = first + (r - *nt * high);
  return true;
}

template <typename T, int MI, int NI, bool AC, bool BC, bool DUAL>
__device__ __forceinline__ void gemm_tile(const GemmOp &g) {
  constexpr int ES = sizeof(T), KB = 64 / ES, NS = 4;
  constexpr int TM = 64 * MI, TN = 64 * NI;
  constexpr int UA = TM / 16, UB = TN / 16;    // 1 KB copy units per stage
  constexpr int VA = UA / 4, VB = UB / 4, VM = VA + VB;          // per wave
  constexpr int SLOT = (TM + TN) * 64;
  constexpr bool SEGS = !AC && BC;             // two contraction segments occur (dx of swiglu)
  static_assert(!DUAL || (!AC && !BC), "the two-matrix product is the forward one");
  static_assert(UA % 4 == 0 && UB % 4 == 0, "units split evenly");
  using OA = Operand<T, AC, TM>;
  using OB = Operand<T, BC, TN>;
  // one LDS object per slot, so that a read of one does not wait for copies
  // into another
  __shared__ __attribute__((aligned(1024))) uint8_t L0[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t L1[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t L2[SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t L3[SLOT];
  uint8_t *const ring[4] = {L0, L1, L2, L3};
  int64_t mt;
  int nt, part;
  if (!gemm_item(g, &mt, &nt, &part)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  constexpr int TO = DUAL ? TN / 2 : TN;       // output columns of a tile
  int half = 0;
  if constexpr (AC) {                          // dW
    const int64_t per = g.m_tiles / g.halves;
    half = mt >= per ? 1 : 0;
    mt -= half * per;
  }
  const int64_t m0 = mt * TM, n0 = (int64_t)nt * TO;

  const int st_seg0 = (int)((g.kdim[0] + KB - 1) / KB);
  const int st_all = SEGS && g.segments > 1 ? st_seg0 + (int)((g.kdim[1] + KB - 1) / KB) : st_seg0;
  const int st_first = (int)((int64_t)st_all * part / g.parts);
  const int nst = (int)((int64_t)st_all * (part + 1) / g.parts) - st_first;

  // sources of the next stage to copy; `rest` counts contraction elements left
  // of its segment for the row operands' ragged ends
  const bool second = SEGS && st_first >= st_seg0;
  const int64_t k_first = (int64_t)(second ? st_first - st_seg0 : st_first) * KB;
  Cursor ca = cursor<T, AC>(second ? g.a[1] : half ? g.a_up : g.a[0], m0, k_first);
  Cursor cb = cursor<T, BC>(second ? g.b[1] : g.b[0], n0, k_first);
  Cursor cu = DUAL ? cursor<T, BC>(g.b_up, n0, k_first) : cb;
  const Cursor ca1 = SEGS ? cursor<T, AC>(g.a[1], m0, 0) : ca;
  const Cursor cb1 = SEGS ? cursor<T, BC>(g.b[1], n0, 0) : cb;
  int to_switch = SEGS && g.segments > 1 && !second ? st_seg0 - st_first : -1;
  int rest = (int)((second ? g.kdim[1] : g.kdim[0]) - k_first), rest_b = rest;
  int to_switch_b = to_switch;
  const int rest1 = (int)g.kdim[1];
  int to_end = nst, to_end_b = nst;            // stages left to copy

  uint32_t off_a[VA], off_b[VB];
#pragma unroll
  for (int q = 0; q < VA; ++q) off_a[q] = OA::source(wave + 4 * q, lane, g.a[0].ld);
#pragma unroll
  for (int q = 0; q < VB; ++q) {
    int u = wave + 4 * q;
    if (DUAL && u >= UB / 2) u -= UB / 2;
    off_b[q] = OB::source(u, lane, g.b[0].ld);
  }
  const int ka = OA::first_k(wave, lane);
  auto copy_a = [&](int slot) {
    rsrc_t r = cursor_rsrc(ca);
    const uint32_t tail = (!AC && ka >= rest) || to_end <= 0 ? kOut : 0u;
#pragma unroll
    for (int q = 0; q < VA; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MOE_LDS void *)(ring[slot] + (wave + 4 * q) * 1024),
                                               16, off_a[q] | tail, 0, 0, 0);
    ca.p += ca.step; ca.left -= ca.step; rest -= KB; --to_end;
    if constexpr (SEGS) {
      const bool sw = --to_switch == 0;
      ca.p = sw ? ca1.p : ca.p; ca.left = sw ? ca1.left : ca.left; rest = sw ? rest1 : rest;
    }
  };
  auto copy_b = [&](int slot) {
    const uint32_t tail = (!BC && ka >= rest_b) || to_end_b <= 0 ? kOut : 0u;
#pragma unroll
    for (int q = 0; q < VB; ++q) {
      const int u = wave + 4 * q;
      // units of the second half hold W_up's rows
      const bool up = DUAL && (UB >= 8 ? q >= VB / 2 : u >= UB / 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(cursor_rsrc(up ? cu : cb), (MOE_LDS void *)(ring[slot] + (UA + u) * 1024), 16,
                                               off_b[q] | tail, 0, 0, 0);
    }
    cb.p += cb.step; cb.left -= cb.step; rest_b -= KB; --to_end_b;
    if constexpr (DUAL) { cu.p += cb.step; cu.left -= cb.step; }
    if constexpr (SEGS) {
      const bool sw = --to_switch_b == 0;
      cb.p = sw ? cb1.p : cb.p; cb.left = sw ? cb1.left : cb.left; rest_b = sw ? rest1 : rest_b;
    }
  };

  f32x16 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  // 32-column block j of the wave; swiglu: the first half of a wave's blocks are
  // gate columns, the rest the up columns that go with them
  auto col_block = [&](int j) {
    return DUAL ? (j < NI / 2 ? wn * (NI / 2) + j : NI + wn * (NI / 2) + j - NI / 2) : wn * NI + j;
  };
  u32x4 fa[2][MI], fb[2][NI];
  auto read = [&](int buf, int slot, int s) {
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[buf][j] = OB::fragment(ring[slot], UA * 1024, col_block(j) * 32, s, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[buf][i] = OA::fragment(ring[slot], 0, (wm * MI + i) * 32, s, lane);
  };
  auto multiply = [&](int buf) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) mma<T>(acc[i][j], fa[buf][i], fb[buf][j]);
  };
  // instructions of a step
  constexpr int kMma = MI * NI * (ES == 2 ? 1 : 4);
  constexpr int kReadsA = MI * (!AC ? 1 : ES == 2 ? 2 : 4);
  constexpr int kReadsB = NI * (!BC ? 1 : ES == 2 ? 2 : 4);

#pragma unroll
  for (int p = 0; p < NS - 1; ++p) { copy_a(p); copy_b(p); }
  __builtin_amdgcn_s_waitcnt(MOE_VMCNT(2 * VM));
  __builtin_amdgcn_s_barrier();
  read(0, 0, 0);
  // Stage st from slot p.  The second step's fragments are read while the first
  // step multiplies; then, with every read of this slot done and the next stage
  // landed (younger: one stage and the A half of another), one barrier, and the
  // next stage's first fragments are read while the second step multiplies.
  // The slot the previous stage used (free since the previous barrier) is
  // refilled meanwhile, A in the first step, B in the second.  Stages past the
  // end copy nothing.
  auto stage = [&](int p) {
    __builtin_amdgcn_sched_barrier(0);
    read(1, p, 1);
    copy_a((p + NS - 1) % NS);
    multiply(0);
    interleave<0, kMma, kReadsA + kReadsB, VA>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(MOE_VMCNT(VM + VA) & ~(15 << 8));   // and lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(0, (p + 1) % NS, 0);
    copy_b((p + NS - 1) % NS);
    multiply(1);
    interleave<0, kMma, kReadsA + kReadsB, VB>();
    __builtin_amdgcn_sched_barrier(0);
  };
  int st = 0;
  for (; st + NS <= nst; st += NS) {
#pragma unroll
    for (int p = 0; p < NS; ++p) stage(p);
  }
#pragma unroll
  for (int p = 0; p < NS - 1; ++p)
    if (st + p < nst) stage(p);
  // Epilogue.  32 rows of the wave's quarter at a time go through the wave's own
  // part of LDS (no barrier), so that a lane then has eight consecutive columns
  // of a row and 16 or 8 lanes a whole line.  bf16: the whole tile's residual is
  // asked for at once, into the registers that the operands have left (in 32-row
  // pieces a read's latency bounded it: 10 % longer at 4096x2048->7168).
  constexpr int NJ = DUAL ? NI / 2 : NI;       // output column blocks of the wave
  constexpr int PC = NJ * 4;                   // pieces of 8 columns per row
  constexpr int PPI = 32 * PC / 64;            // pieces per lane and 32 rows
  constexpr int LD = NI * 32 + 4;              // floats per LDS row (padded)
  constexpr bool RES = !AC && !BC;             // gradients have no residual
  constexpr int AHEAD = RES && ES == 2 ? MI : 1;
  static_assert(32 * LD * 4 <= SLOT, "a wave's rows fit a ring slot");
  float *stage_f = (float *)(wave == 0 ? L0 : wave == 1 ? L1 : wave == 2 ? L2 : L3);
  const bool plain = g.parts > 1;
  // piece q of the wave's rows 32 i ..: row and piece in the block, place in the output
  struct Place {
    int r, pc;
    int64_t m;
    int n;
  };
  auto place = [&](int i, int q) {
    const int idx = q * 64 + lane;
    const int r = idx / PC, pc = idx - r * PC;
    return Place{r, pc, m0 + (wm * MI + i) * 32 + r, (int)n0 + wn * NJ * 32 + pc * 8};
  };
  Raw8<T> res[PPI], ahead[AHEAD][PPI];
  auto fetch = [&](int i, Raw8<T> (&to)[PPI]) {
#pragma unroll
    for (int q = 0; q < PPI; ++q) {
      const Place o = place(i, q);
      if (o.m < g.M && o.n < g.e.N)
        fetch8<T>(to[q], (const T *)g.e.residual + o.m * g.e.ld_res + o.n, g.e.N - o.n,
                  g.e.vec != 0);
    }
  };
  const bool has_res = RES && g.e.residual && !plain;
  Biases<T, DUAL> bias;                        // a lane's columns are the same in every piece
  static_assert(64 % PC == 0, "they are");
  __builtin_amdgcn_s_waitcnt(0);
  if (RES && !plain) bias.fetch(g.e, place(0, 0).n);
  if (AHEAD > 1 && has_res) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(i, ahead[i]);
  }
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();                // every wave is done with the ring
  __builtin_amdgcn_sched_barrier(0);
  for (int ci = 0; ci < MI; ++ci) {
    if (AHEAD == 1 && has_res) fetch(ci, res);
#pragma unroll
    for (int i = 0; i < MI; ++i)
      if (i == ci) {                           // uniform; the accumulators keep their registers
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *(f32x4 *)(stage_f + (lane & 31) * LD + j * 32 + 8 * e + 4 * (lane >> 5)) =
                f32x4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2],
                      acc[i][j][4 * e + 3]};
        if constexpr (AHEAD > 1)
#pragma unroll
          for (int q = 0; q < PPI; ++q) res[q] = ahead[i][q];
      }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < PPI; ++q) {
      const Place o = place(ci, q);
      float v[8], u[8], rs[8];
      load8<float>(v, stage_f + o.r * LD + o.pc * 8, 8, true);
      if constexpr (DUAL) load8<float>(u, stage_f + o.r * LD + NJ * 32 + o.pc * 8, 8, true);
      if (o.m >= g.M || o.n >= g.e.N) continue;
      if (plain) {
        // rows of ldp, a multiple of 8: whole pieces
        float *to =
            g.part + (((int64_t)part * (DUAL ? 2 : g.halves) + half) * g.M + o.m) * g.ldp + o.n;
        store8<float>(to, v, 8, true);
        if constexpr (DUAL) store8<float>(to + g.M * g.ldp, u, 8, true);
      } else if constexpr (!RES) {             // a gradient: no epilogue
        store8<T>((T *)(half ? g.y_up : g.e.y) + o.m * g.e.ld_y + o.n, v, g.e.N - o.n,
                  g.e.vec != 0);
      } else {
        if (has_res) widen8<T>(rs, res[q]);
        finish8<T, DUAL>(g.e, v, u, bias, rs, o.m, o.n);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T, int MI, int NI, bool AC, bool BC, bool DUAL>
__global__ __launch_bounds__(256, MI *NI >= 8 ? 1 : 2) void gemm_kernel(const GemmOp g) {
  gemm_tile<T, MI, NI, AC, BC, DUAL>(g);
}

// Sum of the parts of a split product, in order, and the epilogue.
template <typename T, bool DUAL>
__global__ __launch_bounds__(256) void sum_parts_kernel(const GemmOp g) {
  const int pieces = (g.e.N + 7) / 8;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= g.halves * g.M * pieces) return;
  const int64_t mm = idx / pieces;
  const int n = (int)(idx - mm * pieces) * 8;
  const int half = mm >= g.M ? 1 : 0;
  const int64_t m = mm - half * g.M;
  const int D = DUAL ? 2 : g.halves;
  float v[8] = {}, u[8] = {}, t[8], res[8];
  Biases<T, DUAL> bias;
  bias.fetch(g.e, n);
  if (g.e.residual)
    load8<T>(res, (const T *)g.e.residual + m * g.e.ld_res + n, g.e.N - n, g.e.vec != 0);
  for (int p = 0; p < g.parts; ++p) {
    const float *o = g.part + (((int64_t)p * D + half) * g.M + m) * g.ldp + n;
    load8<float>(t, o, 8, true);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += t[j];
    if constexpr (DUAL) {
      load8<float>(t, o + g.M * g.ldp, 8, true);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += t[j];
    }
  }
  Epilogue e = g.e;
  if (half) e.y = g.y_up;
  finish8<T, DUAL>(e, v, u, bias, res, m, n);
}

// ---------------------------------------------------------------------------
// Rows of `cols` elements at stride ld to padded rows of ldo, zeros behind.
template <typename T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const T *src, int64_t ld, int64_t rows,
                                                       int cols, T *dst, int64_t ldo) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t pieces = ldo / (16 / sizeof(T));
  if (idx >= rows * pieces) return;
  const int64_t r = idx / pieces;
  const int c = (int)(idx - r * pieces) * (int)(16 / sizeof(T));
  alignas(16) T v[16 / sizeof(T)];
#pragma unroll
  for (int j = 0; j < (int)(16 / sizeof(T)); ++j)
    v[j] = c + j < cols ? src[r * ld + c + j] : (T)0.f;
  *(u32x4 *)(dst + r * ldo + c) = *(const u32x4 *)v;
}

// dz = dy act'(z) (swiglu: dz and du) in rows of ldz, zeros behind column N,
// and the column sums of dz over this workgroup's rows.  A workgroup takes 64
// columns and a share of the rows: thread (c8, r) eight columns of every 32nd row.
struct SlopeArgs {
  const void *dy, *z, *z_up;
  void *dz, *du;               // null: column sums alone
  float *sums;                 // [parts][DUAL ? 2 : 1][N], or null
  int64_t M, ld_dy, ldz;
  int N, act, parts, vec;
  float limit;
};
template <typename T, bool DUAL>
__global__ __launch_bounds__(256) void slope_kernel(const SlopeArgs a) {
  constexpr int D = DUAL ? 2 : 1;
  __shared__ float red[D][32][65];
  const int c8 = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int n = blockIdx.x * 64 + c8 * 8;
  const int part = blockIdx.y;
  const int64_t lo = a.M * part / a.parts, hi = a.M * (part + 1) / a.parts;
  const int left = a.N - n;
  const bool vec = a.vec != 0;
  float s[D][8] = {};
  // a row's loads are under way while the one before is finished
  Raw8<T> ng = {}, nz = {}, nu = {};
  auto fetch = [&](int64_t m) {
    if (left <= 0 || m >= hi) return;
    fetch8<T>(ng, (const T *)a.dy + m * a.ld_dy + n, left, vec);
    if (a.z) fetch8<T>(nz, (const T *)a.z + m * a.N + n, left, vec);
    if constexpr (DUAL) fetch8<T>(nu, (const T *)a.z_up + m * a.N + n, left, vec);
  };
  fetch(lo + r0);
  for (int64_t m = lo + r0; m < hi; m += 32) {
    float g[8], z[8], u[8], dz[8], du[8];
    if (left <= 0 && n >= a.ldz) break;
    widen8<T>(g, ng);
    widen8<T>(z, nz);
    if constexpr (DUAL) widen8<T>(u, nu);
    fetch(m + 32);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // `none` has slope 1 for any z
      dz[j] = du[j] = 0.f;
      if (j < left) grad_of<T, DUAL>(g[j], z[j], u[j], a.act, a.limit, &dz[j], &du[j]);
      s[0][j] += dz[j];
      if constexpr (DUAL) s[1][j] += du[j];
    }
    if (a.dz && n < a.ldz) {
      store8<T>((T *)a.dz + m * a.ldz + n, dz, (int)(a.ldz - n < 8 ? a.ldz - n : 8), true);
      if constexpr (DUAL)
        store8<T>((T *)a.du + m * a.ldz + n, du, (int)(a.ldz - n < 8 ? a.ldz - n : 8), true);
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int d = 0; d < D; ++d)
#pragma unroll
    for (int j = 0; j < 8; ++j) red[d][r0][c8 * 8 + j] = s[d][j];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * D; i += 256) {
    const int d = i >> 6, c = i & 63;
    if (blockIdx.x * 64 + c >= a.N) continue;
    float v = 0.f;
    for (int r = 0; r < 32; ++r) v += red[d][r][c];
    a.sums[((int64_t)part * D + d) * a.N + blockIdx.x * 64 + c] = v;
  }
}

// db: the parts' column sums.  A workgroup takes 32 columns, eight threads each
// a column's parts p, p + 8, ... (loads that do not wait for one another), added
// in a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void bias_sum_kernel(const float *sums, int N, int parts, int d,
                                                       T *db, T *db_up) {
  __shared__ float red[8][33];
  const int c = threadIdx.x & 31, p0 = threadIdx.x >> 5, which = blockIdx.y;
  const int n = blockIdx.x * 32 + c;
  float v = 0.f;
  if (n < N)
#pragma unroll 4
    for (int p = p0; p < parts; p += 8) v += sums[((int64_t)p * d + which) * N + n];
  red[p0][c] = v;
  __syncthreads();
  T *out = which ? db_up : db;
  if (p0 || n >= N || !out) return;
  v = 0.f;
#pragma unroll
  for (int p = 0; p < 8; ++p) v += red[p][c];
  out[n] = (T)v;
}

// ---------------------------------------------------------------------------
// Tile shape and parts of a product of `rows` x `cols` (cols of both matrices
// for swiglu) over `stages` stages: the one with the least estimated time.
//
// One workgroup a CU and round; a round costs its stages and a fixed part (first
// copies, epilogue).  The constants are microseconds measured over products of
// 1024..8192 a side, one shape forced at a time (bf16 4096x4096 over K = 1024,
// 2048, 4096: 256x256 tiles 44, 69, 121 us, 256x128 52, 85, 150, 128x128 46, 85,
// 165, 64x64 67, 134, 271; dx and dW of that size within 10% of these).  A bf16
// round that fills part of the GPU runs at a higher clock (4096x2048 over K =
// 4096 with 128 tiles of 256x256: 105 us).  `alone`: a stage of a workgroup that
// has its CU to itself, where that is longer (one chain of MFMAs and reads).
struct Shape {
  int mi, ni, parts;
  double us;                   // the estimate
};

Shape pick_shape(int64_t rows, int64_t cols, int64_t stages, bool f32, bool dual) {
  struct Cost { int mi, ni; double stage, alone, fixed; };
  const Cost in_bf16[] = {{4, 4, 0.80, 0.56, 14.0},
                          {4, 2, 0.52, 0.36, 8.0},
                          {2, 2, 0.27, 0.22, 3.5},
                          {1, dual ? 2 : 1, dual ? 0.186 : 0.127, 0.2, 1.0}};
  // fp32 MFMAs bound every shape alike (256x256 3.8 a stage and 14 fixed, 256x128
  // 1.9 and 8): the larger tiles are at best as fast, and there are none
  const Cost in_f32[] = {{2, 2, 0.94, 0.94, 3.5},
                         {1, dual ? 2 : 1, dual ? 0.5 : 0.254, dual ? 0.6 : 0.33, 1.0}};
  const Cost *shapes = f32 ? in_f32 : in_bf16;
  Shape best = {1, 1, 1, 1e300};
  for (int i = 0; i < (f32 ? 2 : 4); ++i) {
    const Cost &sh = shapes[i];
    const int64_t tiles = ((rows + 64 * sh.mi - 1) / (64 * sh.mi)) *
                          ((cols + 64 * sh.ni - 1) / (64 * sh.ni));
    for (int parts = 1; parts <= 16; parts *= 2) {
      if (parts > 1 && (stages < 16 * parts || tiles * parts > 1024)) break;
      const int64_t items = tiles * parts, full = items / 256;
      const double last = (double)(items - full * 256) / 256;
      const double deep = (double)((stages + parts - 1) / parts);
      double t = full * (deep * sh.stage + sh.fixed);
      if (last > 0) {
        const double s = f32 ? sh.stage : sh.stage * (0.7 + 0.3 * last);
        t += deep * (full == 0 && sh.alone > s ? sh.alone : s) + sh.fixed;
      }
      // partial sums: a launch, and written and read at 8 TB/s in all
      if (parts > 1) t += 5.0 + (double)rows * cols * parts * 1e-6;
      if (t < best.us) best = {sh.mi, sh.ni, parts, t};
    }
  }
  return best;
}

Shape shape_of(int64_t rows, int64_t cols, const int64_t *kdim, int segments, int dtype,
               bool dual) {
  const int64_t kb = dtype == MOE_DTYPE_F32 ? 16 : 32;
  int64_t st = 0;
  for (int i = 0; i < segments; ++i) st += (kdim[i] + kb - 1) / kb;
  return pick_shape(rows, cols, st, dtype == MOE_DTYPE_F32, dual);
}

size_t part_bytes(int64_t rows, int64_t cols, bool dual, const Shape &s) {
  return s.parts > 1 ? (size_t)s.parts * (dual ? 2 : 1) * rows * ((cols + 7) / 8 * 8) * 4 : 0;
}

template <typename T, int MI, int NI, bool AC, bool BC, bool DUAL>
hipError_t run_gemm_shape(GemmOp g, hipStream_t s) {
  constexpr int TM = 64 * MI, TO = DUAL ? 32 * NI : 64 * NI;
  g.m_tiles = (g.M + TM - 1) / TM * g.halves;
  g.n_tiles = (g.e.N + TO - 1) / TO;
  const int64_t items = g.m_tiles * g.n_tiles * g.parts;
  hipLaunchKernelGGL((gemm_kernel<T, MI, NI, AC, BC, DUAL>), dim3((unsigned)(8 * ((items + 7) / 8))),
                     dim3(256), 0, s, g);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || g.parts == 1) return err;
  const int64_t pieces = g.halves * g.M * ((g.e.N + 7) / 8);
  hipLaunchKernelGGL((sum_parts_kernel<T, DUAL>), dim3((unsigned)((pieces + 255) / 256)), dim3(256),
                     0, s, g);
  return hipGetLastError();
}

template <typename T, bool AC, bool BC, bool DUAL>
hipError_t run_gemm(GemmOp g, const Shape &sh, void *part, hipStream_t s) {
  g.parts = sh.parts;
  if (g.halves < 1) g.halves = 1;
  g.part = (float *)part;
  g.ldp = (g.e.N + 7) / 8 * 8;
  if constexpr (sizeof(T) == 2) {
    if (sh.mi == 4 && sh.ni == 4) return run_gemm_shape<T, 4, 4, AC, BC, DUAL>(g, s);
    if (sh.mi == 4) return run_gemm_shape<T, 4, 2, AC, BC, DUAL>(g, s);
  }
  if (sh.mi == 2) return run_gemm_shape<T, 2, 2, AC, BC, DUAL>(g, s);
  return run_gemm_shape<T, 1, DUAL ? 2 : 1, AC, BC, DUAL>(g, s);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Tile shape and parts of a product of a call, wherever they are asked for.
Shape product_shape(const moe_linear_config &c, int32_t product) {
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim, kd[2] = {N, N};
  const bool dual = c.activation == MOE_ACTIVATION_SWIGLU;
  if (product == MOE_LINEAR_FORWARD) return shape_of(M, dual ? 2 * N : N, &K, 1, c.dtype, dual);
  if (product == MOE_LINEAR_DX) return shape_of(M, K, kd, dual ? 2 : 1, c.dtype, false);
  return shape_of(dual ? 2 * N : N, K, &M, 1, c.dtype, false);
}

// The kernels of a call.  Up to kFewRows rows take the stream of W where no copy
// has to be made first (1x7168->2x2048 swiglu bf16 11.4 us, 17.5 by tiles;
// 16x4096->4096 fp32 18, 29 by tiles).  Otherwise 32 x 32 tiles where their estimate is below that
// of the GEMM with the launches around it (4 us each, with the wait for the one
// before).  Microseconds per round of 256 tiles and eight chunks of the
// contraction, measured with either way forced on 60 shapes: 203x777->1023 fp32
// 30 by the GEMM and 12 by small tiles, 64x4096->512 18 and 28, 1024^3 26 and 36;
// the backward of 301x256->320 29 and 16, of 1024^3 61 and 148.
double small_us(int64_t tiles, int64_t contraction, double chunks_us) {
  const int64_t chunks = (contraction + 63) / 64;
  return (double)tiles / 256 * (2.0 + (double)((chunks + 7) / 8) * chunks_us);
}

moe_linear_path_kind forward_path(const moe_linear_config &c) {
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim;
  const bool dual = c.activation == MOE_ACTIVATION_SWIGLU;
  const bool copy_w = linear_odd_rows(K, K, c.dtype), copy_x = linear_odd_rows(K, c.ld_x, c.dtype);
  if (M <= kFewRows && !copy_w && !copy_x) return MOE_LINEAR_PATH_FEW;
  const Shape sh = product_shape(c, MOE_LINEAR_FORWARD);
  const double gemm = sh.us + 4.0 * (1 + copy_x + copy_w * (dual ? 2 : 1));
  const int64_t tiles = (M + 31) / 32 * ((N + 31) / 32);
  const double small = small_us((tiles + 255) / 256 * 256, K, dual ? 5.2 : 3.0) + 4.0;
  return small < gemm ? MOE_LINEAR_PATH_SMALL : MOE_LINEAR_PATH_TILED;
}

// By the time of all gradients, whichever are asked for: each comes out the same
// alone and with others.
bool backward_small(const moe_linear_config &c) {
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim;
  if (M == 0) return false;
  const bool dual = c.activation == MOE_ACTIVATION_SWIGLU;
  const double chunks_us = dual ? 9.0 : 7.0;
  const int64_t kt = (K + 31) / 32, both = dual ? 2 : 1;
  const Shape dx = product_shape(c, MOE_LINEAR_DX), dw = product_shape(c, MOE_LINEAR_DW);
  // slope, column sums, products and copies
  const double gemm = 16.0 + dx.us + dw.us + (linear_odd_rows(K, K, c.dtype) ? 4.0 * both : 0.0) +
                      (linear_odd_rows(K, c.ld_x, c.dtype) ? 4.0 : 0.0);
  // the workgroups of dx and dW fill the GPU together
  double small = small_us((M + 31) / 32 * kt, both * N, chunks_us) +
                 small_us((N + 31) / 32 * kt * both, M, chunks_us);
  for (const int64_t chain : {both * N, M}) {
    const double one = small_us(256, chain, chunks_us);
    small = small > one ? small : one;
  }
  return small + 4.0 < gemm;
}

template <typename T>
hipError_t pad_rows(const void *src, int64_t ld, int64_t rows, int cols, void *dst, int64_t ldo,
                    hipStream_t s) {
  const int64_t n = rows * (ldo / (16 / sizeof(T)));
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL((pad_rows_kernel<T>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     (const T *)src, ld, rows, cols, (T *)dst, ldo);
  return hipGetLastError();
}

// Row chunks of the column sums: enough workgroups to fill the GPU, each with
// rows to add.
int colsum_parts(int64_t M, int N) {
  const int64_t across = (N + 63) / 64;
  int64_t parts = (1024 + across - 1) / across;
  const int64_t most = (M + 63) / 64;
  return (int)(parts > most ? most : parts);
}

template <typename T>
hipError_t linear_forward(const moe_linear_config &c, const moe_linear_weights &w, const void *x,
                          const void *residual, void *y, void *z, void *z_up, char *ws,
                          hipStream_t s) {
  const LinearSpace L = linear_space(c, false, false, false, false);
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim;
  const bool dual = c.activation == MOE_ACTIVATION_SWIGLU;
  Epilogue e = {};
  e.bias = w.bias; e.bias_up = w.bias_up; e.residual = residual;
  e.y = y; e.z = z; e.z_up = z_up;
  e.ld_y = c.ld_y; e.ld_res = c.ld_residual; e.ld_z = N;
  e.N = (int)N; e.act = c.activation; e.limit = c.limit;
  e.vec = !linear_odd_rows(N, c.ld_y, c.dtype) && (!residual || !linear_odd_rows(N, c.ld_residual, c.dtype)) &&
          N % 8 == 0 && aligned16(y) && aligned16(z) && aligned16(z_up) && aligned16(residual) &&
          aligned16(w.bias) && aligned16(w.bias_up);
  const moe_linear_path_kind path = forward_path(c);
  if (path != MOE_LINEAR_PATH_TILED) {
    SmallArgs a = {};
    a.x = x; a.w = w.w; a.w_up = w.w_up;
    a.M = M; a.K = K; a.ld_x = c.ld_x;
    a.e = e;
    return path == MOE_LINEAR_PATH_FEW ? launch_few_rows<T>(a, dual, s)
                                       : launch_small_forward<T>(a, dual, s);
  }
  hipError_t err;
  Matrix mx = {x, c.ld_x, M, K}, mw = {w.w, K, N, K}, mu = {w.w_up, K, N, K};
  const int64_t Kp = linear_pad(K, c.dtype);
  if (linear_odd_rows(K, c.ld_x, c.dtype)) {
    if ((err = pad_rows<T>(x, c.ld_x, M, (int)K, ws + L.x, Kp, s)) != hipSuccess) return err;
    mx = {ws + L.x, Kp, M, Kp};
  }
  if (linear_odd_rows(K, K, c.dtype)) {
    if ((err = pad_rows<T>(w.w, K, N, (int)K, ws + L.w, Kp, s)) != hipSuccess) return err;
    mw = {ws + L.w, Kp, N, Kp};
    if (dual) {
      if ((err = pad_rows<T>(w.w_up, K, N, (int)K, ws + L.w_up, Kp, s)) != hipSuccess) return err;
      mu = {ws + L.w_up, Kp, N, Kp};
    }
  }
  GemmOp g = {};
  g.a[0] = mx; g.b[0] = mw; g.b_up = mu;
  g.kdim[0] = K;
  g.segments = 1;
  g.M = M;
  g.e = e;
  const Shape sh = product_shape(c, MOE_LINEAR_FORWARD);
  return dual ? run_gemm<T, false, false, true>(g, sh, ws + L.part, s)
              : run_gemm<T, false, false, false>(g, sh, ws + L.part, s);
}

template <typename T>
hipError_t linear_backward(const moe_linear_config &c, const moe_linear_weights &w, const void *x,
                           const void *dy, const void *z, const void *z_up,
                           const moe_linear_grads &gr, char *ws, hipStream_t s) {
  const bool dual = c.activation == MOE_ACTIVATION_SWIGLU;
  const bool want_dw = gr.dw || gr.dw_up, want_db = gr.dbias || gr.dbias_up;
  const LinearSpace L = linear_space(c, true, gr.dx != nullptr, want_dw, want_db);
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim;
  const int64_t Kp = linear_pad(K, c.dtype), Np = linear_pad(N, c.dtype);
  hipError_t err;
  if (backward_small(c)) {
    SmallArgs a = {};
    a.x = x; a.w = w.w; a.w_up = w.w_up;
    a.dy = dy; a.z = c.activation == MOE_ACTIVATION_NONE ? nullptr : z; a.z_up = z_up;
    a.dx = gr.dx; a.dw = gr.dw; a.dw_up = gr.dw_up; a.db = gr.dbias; a.db_up = gr.dbias_up;
    a.M = M; a.K = K; a.ld_x = c.ld_x; a.ld_dy = c.ld_y; a.ld_dx = gr.ld_dx;
    a.e.N = (int)N; a.e.act = c.activation; a.e.limit = c.limit;
    return launch_small_backward<T>(a, dual, s);
  }
  // dz: dy itself where nothing changes it and its rows are whole pieces
  const bool same = c.activation == MOE_ACTIVATION_NONE && !linear_odd_rows(N, c.ld_y, c.dtype);
  Matrix mz = {dy, c.ld_y, M, N}, mu = {};
  if (!same) {
    mz = {ws + L.dz, Np, M, Np};
    if (dual) mu = {ws + L.du, Np, M, Np};
  }
  if (!same || want_db) {
    SlopeArgs a = {};
    a.dy = dy; a.z = c.activation == MOE_ACTIVATION_NONE ? nullptr : z; a.z_up = z_up;
    a.dz = same || !(gr.dx || want_dw) ? nullptr : ws + L.dz;
    a.du = ws + L.du;
    a.sums = want_db ? (float *)(ws + L.colsum) : nullptr;
    a.M = M; a.ld_dy = c.ld_y; a.ldz = Np; a.N = (int)N; a.act = c.activation;
    a.limit = c.limit;
    a.parts = colsum_parts(M, (int)N);
    a.vec = !linear_odd_rows(N, c.ld_y, c.dtype) && N % 8 == 0 && aligned16(z) && aligned16(z_up);
    const dim3 grid((unsigned)((Np + 63) / 64), (unsigned)a.parts);
    if (M > 0) {                               // no rows: the sums below are empty
      if (dual) hipLaunchKernelGGL((slope_kernel<T, true>), grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((slope_kernel<T, false>), grid, dim3(256), 0, s, a);
    }
    if ((err = hipGetLastError()) != hipSuccess) return err;
    if (want_db) {
      const int d = dual ? 2 : 1;
      hipLaunchKernelGGL((bias_sum_kernel<T>), dim3((unsigned)((N + 31) / 32), (unsigned)d),
                         dim3(256), 0, s, (const float *)(ws + L.colsum), (int)N, a.parts, d, (T *)gr.dbias,
                         (T *)gr.dbias_up);
      if ((err = hipGetLastError()) != hipSuccess) return err;
    }
  }
  if (gr.dx && M > 0) {
    Matrix mw = {w.w, K, N, K}, mwu = {w.w_up, K, N, K};
    if (linear_odd_rows(K, K, c.dtype)) {
      if ((err = pad_rows<T>(w.w, K, N, (int)K, ws + L.w, Kp, s)) != hipSuccess) return err;
      mw = {ws + L.w, Kp, N, Kp};
      if (dual) {
        if ((err = pad_rows<T>(w.w_up, K, N, (int)K, ws + L.w_up, Kp, s)) != hipSuccess) return err;
        mwu = {ws + L.w_up, Kp, N, Kp};
      }
    }
    GemmOp g = {};
    g.a[0] = mz; g.b[0] = mw;
    g.a[1] = mu; g.b[1] = mwu;
    g.kdim[0] = N; g.kdim[1] = N;
    g.segments = dual ? 2 : 1;
    g.M = M;
    g.e.y = gr.dx; g.e.ld_y = gr.ld_dx; g.e.N = (int)K; g.e.act = MOE_ACTIVATION_NONE;
    g.e.vec = !linear_odd_rows(K, gr.ld_dx, c.dtype) && K % 8 == 0 && aligned16(gr.dx);
    const Shape sh = product_shape(c, MOE_LINEAR_DX);
    if ((err = run_gemm<T, false, true, false>(g, sh, ws + L.part, s)) != hipSuccess) return err;
  }
  if (want_dw) {
    Matrix mx = {x, c.ld_x, M, K};
    if (linear_odd_rows(K, c.ld_x, c.dtype)) {
      if ((err = pad_rows<T>(x, c.ld_x, M, (int)K, ws + L.x, Kp, s)) != hipSuccess) return err;
      mx = {ws + L.x, Kp, M, Kp};
    }
    // both products of swiglu in one launch, or the one that is wanted
    const bool both = gr.dw && gr.dw_up;
    GemmOp g = {};
    g.a[0] = gr.dw ? mz : mu; g.b[0] = mx;
    g.a_up = mu; g.y_up = gr.dw_up;
    g.halves = both ? 2 : 1;
    g.kdim[0] = M;
    g.segments = 1;
    g.M = N;
    g.e.y = gr.dw ? gr.dw : gr.dw_up; g.e.ld_y = K; g.e.N = (int)K;
    g.e.act = MOE_ACTIVATION_NONE;
    g.e.vec = K % 8 == 0 && aligned16(gr.dw) && aligned16(gr.dw_up);
    const Shape sh = product_shape(c, MOE_LINEAR_DW);
    if ((err = run_gemm<T, true, true, false>(g, sh, ws + L.part, s)) != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace

LinearSpace linear_space(const moe_linear_config &c, bool backward, bool dx, bool dw, bool db) {
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim;
  const int64_t Kp = linear_pad(K, c.dtype), Np = linear_pad(N, c.dtype);
  const size_t es = c.dtype == MOE_DTYPE_F32 ? 4 : 2;
  const bool dual = c.activation == MOE_ACTIVATION_SWIGLU;
  LinearSpace l = {};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  // what the GEMM takes, also where another kernel runs: one size per shape
  const bool use_x = !backward || dw, use_w = !backward || dx;
  l.x = take(use_x && linear_odd_rows(K, c.ld_x, c.dtype) ? es * M * Kp : 0);
  l.w = take(use_w && linear_odd_rows(K, K, c.dtype) ? es * N * Kp : 0);
  l.w_up = take(use_w && dual && linear_odd_rows(K, K, c.dtype) ? es * N * Kp : 0);
  size_t part = 0;
  auto need = [&](int64_t rows, int64_t cols, bool two, int32_t product) {
    const size_t b = part_bytes(rows, cols, two, product_shape(c, product));
    if (b > part) part = b;
  };
  if (backward) {
    const bool same = c.activation == MOE_ACTIVATION_NONE && !linear_odd_rows(N, c.ld_y, c.dtype);
    l.dz = take(!same && (dx || dw) ? es * M * Np : 0);
    l.du = take(dual && (dx || dw) ? es * M * Np : 0);
    l.colsum = take(db ? sizeof(float) * colsum_parts(M, (int)N) * (dual ? 2 : 1) * N : 0);
    if (dx) need(M, K, false, MOE_LINEAR_DX);
    if (dw) need(dual ? 2 * N : N, K, false, MOE_LINEAR_DW);
  } else {
    need(M, N, dual, MOE_LINEAR_FORWARD);
  }
  l.part = take(part);
  l.total = off;
  return l;
}

moe_linear_path_info linear_path(const moe_linear_config &c, int32_t product) {
  moe_linear_path_info info = {};
  if (product == MOE_LINEAR_FORWARD) info.path = forward_path(c);
  else if (backward_small(c)) info.path = MOE_LINEAR_PATH_SMALL;
  if (info.path != MOE_LINEAR_PATH_TILED) return info;
  const Shape s = product_shape(c, product);
  info.tile_rows = 64 * s.mi;
  info.tile_cols = 64 * s.ni;
  info.parts = s.parts;
  return info;
}

bool linear_launchable(const moe_linear_config &c, bool backward) {
  const int64_t M = c.rows, K = c.in_dim, N = c.out_dim, wide = K > N ? K : N;
  // at most one thread an element, in tiles of 32 x 32 (512 threads): most calls
  if ((M + 32) * (wide + 32) < (int64_t)1 << 31 && (N + 32) * (K + 32) < (int64_t)1 << 30) return true;
  const int64_t both = c.activation == MOE_ACTIVATION_SWIGLU ? 2 : 1;
  auto tiles = [](int64_t rows, int64_t cols, int64_t r, int64_t q) {
    return (rows + r - 1) / r * ((cols + q - 1) / q);
  };
  int64_t most = 0;
  auto launch = [&](int64_t threads) { most = threads > most ? threads : most; };
  // the two matrices of swiglu's forward share a tile, those of its dW do not
  auto gemm = [&](int64_t rows, int64_t cols, int32_t product) {
    const Shape s = product_shape(c, product);
    const int64_t wide = 64 * s.ni / (product == MOE_LINEAR_FORWARD ? both : 1);
    const int64_t n = tiles(rows, cols, 64 * s.mi, wide) * (product == MOE_LINEAR_DW ? both : 1);
    launch(256 * ((n * s.parts + 7) / 8 * 8));
  };
  const int64_t pieces = (K + linear_pad(1, c.dtype) - 1) / linear_pad(1, c.dtype);
  if (backward && backward_small(c)) {
    launch(512 * (tiles(M, K, 32, 32) + both * tiles(N, K, 32, 32)));
  } else if (backward) {
    gemm(M, K, MOE_LINEAR_DX);
    gemm(N, K, MOE_LINEAR_DW);
  } else if (const auto path = forward_path(c); path == MOE_LINEAR_PATH_SMALL) {
    launch(512 * tiles(M, N, 32, 32));
  } else if (path == MOE_LINEAR_PATH_TILED) {
    gemm(M, N, MOE_LINEAR_FORWARD);
  }
  if (linear_odd_rows(K, c.ld_x, c.dtype)) launch(M * pieces + 256);
  if (linear_odd_rows(K, K, c.dtype)) launch(N * pieces + 256);
  return most < (int64_t)1 << 32;
}

hipError_t launch_linear(const moe_linear_config &c, const moe_linear_weights &w, const void *x,
                         const void *residual, void *y, void *z, void *z_up, char *ws,
                         hipStream_t s) {
  return c.dtype == MOE_DTYPE_F32
             ? linear_forward<float>(c, w, x, residual, y, z, z_up, ws, s)
             : linear_forward<bf16>(c, w, x, residual, y, z, z_up, ws, s);
}

hipError_t launch_linear_backward(const moe_linear_config &c, const moe_linear_weights &w,
                                  const void *x, const void *dy, const void *z, const void *z_up,
                                  const moe_linear_grads &g, char *ws, hipStream_t s) {
  return c.dtype == MOE_DTYPE_F32 ? linear_backward<float>(c, w, x, dy, z, z_up, g, ws, s)
                                  : linear_backward<bf16>(c, w, x, dy, z, z_up, g, ws, s);
}

}  // namespace moe
