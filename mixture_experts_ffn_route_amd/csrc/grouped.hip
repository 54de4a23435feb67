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
// Where an expert's rows begin is known on the device alone: every workgroup scans
// the offsets once (a wave's prefix sum over the experts' tiles) and finds its tiles by
// that, so nothing waits for a list.  Offsets are clamped to [0, rows], and an expert that
// ends before it starts has no rows, so whatever they hold no access is out of range.
// (After such a descent an expert's rows can be another's too, and its results either's.)
//
// Workgroups are as many as the GPU holds at once and walk their tiles one after
// another: starting a workgroup for every tile left 2.6 us between one's end and the
// next one's first instruction, and 2 us of scan, in 15 us a tile of the weight
// gradients.

#include <type_traits>

#include "keep.h"
#include "tile.h"
#include "train.h"
#include "walk.h"

namespace moe {
namespace {

struct GroupedOp {
  GemmOp g;                    // pointers of expert 0 and row 0
  const int32_t *offsets;
  int64_t rows;
  int E;
  int64_t b_expert;            // bytes from one expert's B (weights) to the next's
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

// One tile: rows m0 .. of the expert's, its height in blocks of 64 rows, the column
// tile.
struct GroupedItem {
  int e, lo, n;                // expert, its first row and rows
  int m0, blocks;
  int nt, half;                // half: of the second matrix
};

// Tiles of up to HIGH blocks of 64 rows that cover n rows, of as equal heights as
// blocks allow, so that none is nearly empty.
template <int HIGH>
__device__ __forceinline__ int tiles_of(int n) { return ((n + 63) / 64 + HIGH - 1) / HIGH; }
__device__ __forceinline__ void height_of(int blocks, int tiles, int i, GroupedItem *out) {
  const int low = blocks / tiles, higher = blocks - low * tiles;
  out->m0 = (i * low + (i < higher ? i : higher)) * 64;
  out->blocks = low + (i < higher ? 1 : 0);
}

// What the experts before each lane's own amount to (a lane has E / 64 of them, one
// after another), and the expert that a position falls to.
template <class N, class F>
struct Line {
  const F size;                // of an expert
  const int E, chunk;
  N mine, upto;                // of this lane's experts, and with those before them
  __device__ __forceinline__ Line(int experts, F f) : size(f), E(experts), chunk((experts + 63) / 64) {
    const int lane = threadIdx.x & 63;
    mine = 0;
    for (int i = 0; i < chunk; ++i)
      if (lane * chunk + i < E) mine += size(lane * chunk + i);
    upto = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const N o = __shfl_up(upto, off);
      if (lane >= off) upto += o;
    }
  }
  static __device__ __forceinline__ N of_lane(N v, int lane) {
    if constexpr (sizeof(N) == 4) {
      return __builtin_amdgcn_readlane(v, lane);
    } else {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
      return (N)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 | lo);
    }
  }
  __device__ __forceinline__ N total() const { return of_lane(upto, 63); }
  // The expert at `pos` < total(), and where it starts.
  __device__ __forceinline__ int at(N pos, N *start) const {
    const int lane = threadIdx.x & 63;
    const int src = __ffsll((unsigned long long)__ballot(upto > pos)) - 1;
    N from = upto - mine;
    int e = lane * chunk;
    if (chunk > 1 && lane == src)
      for (; e < E - 1; ++e) {
        const N n = size(e);
        if (pos < from + n) break;
        from += n;
      }
    *start = of_lane(from, src);
    return __builtin_amdgcn_readlane(e, src);
  }
};
template <class N, class F>
__device__ __forceinline__ Line<N, F> line_of(int experts, F f) { return Line<N, F>(experts, f); }

template <typename T>
__device__ __forceinline__ void move(Matrix &m, const GroupedItem &it) {
  m.p = (const T *)m.p + (int64_t)it.lo * m.ld;
  m.rows = it.n;
}

// ---------------------------------------------------------------------------
// Endings.  Stores (and loads) are buffer ones without a branch, past the tile's rows
// or the matrix's columns at an offset that drops them (reads zeros), so that a load's
// wait does not have to be one for all stores before it.

// The nontemporal policy: of results, and of weights that one or two row tiles read, by
// columns (whole lines at a time), so that they leave the caches to the rows that tiles
// share.  8192 rows of 48 experts, 5120 -> 2 x 1536: all six products 2267 us, the
// results so 2136, the weights of dh and dx too 2015.  Weights read by rows come half a line
// a stage, and such a line is gone before its other half is needed (up 215, so 234).
constexpr int kStream = 2;

// Rows that a tile reads or writes, from its first.
__device__ __forceinline__ int height(int left, int high) { return left < high ? left : high; }
__device__ __forceinline__ rsrc_t rows_rsrc(const void *p, int64_t first, int rows, int64_t row_bytes) {
  const uint8_t *at = (const uint8_t *)p + first * row_bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(at), 0, (uint32_t)(rows * row_bytes),
                                           0x00027000);
}

// Eight columns of type T at byte `off`, of which `left` are in the matrix (whole
// pieces of 16 bytes).
template <typename T>
__device__ __forceinline__ void store_piece(rsrc_t r, uint32_t off, const float (&v)[8], int left) {
  if constexpr (sizeof(T) == 2) {
    bf16x8 b;
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = (bf16)v[j];
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, b), r, left > 0 ? off : kOut, 0, 0);
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{__float_as_uint(v[4 * p]), __float_as_uint(v[4 * p + 1]), __float_as_uint(v[4 * p + 2]),
                __float_as_uint(v[4 * p + 3])},
          r, left > 4 * p ? off + 16 * p : kOut, 0, 0);
  }
}
template <typename T>
__device__ __forceinline__ void fetch_piece(Raw8<T> &a, rsrc_t r, uint32_t off, int left) {
#pragma unroll
  for (int p = 0; p < (int)sizeof(T) / 2; ++p) {
    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(
        r, left > p * (16 / (int)sizeof(T)) ? off + 16 * p : kOut, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) a.w[4 * p + j] = w[j];
  }
}

// Rows of sums, rounded: y and dx; the weight gradients.
template <typename T>
struct SumsOut {
  static constexpr bool sums = true;
  struct Tile {
    rsrc_t y;
  };
  T *y, *y_up;                 // y_up: of the second matrix
  int N, M;                    // M > 0: rows of every expert's matrix
  __device__ __forceinline__ Tile begin(const GroupedItem &it, int high) const {
    const int64_t first = (M ? (int64_t)it.e * M : it.lo) + it.m0;
    return Tile{rows_rsrc(it.half ? y_up : y, first, height((M ? M : it.n) - it.m0, high),
                          (int64_t)N * sizeof(T))};
  }
  __device__ __forceinline__ void put(const Tile &t, int m, int n, const u32x4 &piece) const {
    __builtin_amdgcn_raw_buffer_store_b128(piece, t.y, n < N ? ((uint32_t)m * N + n) * sizeof(T) : kOut, 0,
                                           kStream);
  }
};

// Eight values of z or u in 8 bits: the four neighbouring lanes hold a block.
__device__ __forceinline__ void keep_piece(const float (&v)[8], float limit, rsrc_t codes, rsrc_t scales,
                                           uint32_t at, uint32_t block, bool on, bool first) {
  float m = keep_top_of_sums(v);
  m = fmaxf(m, xor_lane<1>(m));
  m = fmaxf(m, xor_lane<2>(m));
  const int X = keep_exponent(m);
  uint32_t c[2];
  keep<8>(v, X, limit, c);
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{c[0], c[1]}, codes, on ? at : kOut, 0, 0);
  __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(X + 127), scales, on && first ? block : kOut, 0, 0);
}

// Saved z and u of a tile's rows.
struct SavedTile {
  rsrc_t z, u, zs, us;
  __device__ __forceinline__ SavedTile(const moe_experts_saved &s, int64_t first, int rows, int N) {
    const int64_t bytes = s.kind == MOE_SAVE_NONE ? 0 : s.kind == MOE_SAVE_MXFP8 ? N : N * (int64_t)4;
    const int64_t scales = s.kind == MOE_SAVE_MXFP8 ? N / 32 : 0;
    z = rows_rsrc(s.gate, first, rows, bytes);
    u = rows_rsrc(s.up, first, rows, bytes);
    zs = rows_rsrc(s.gate_scales, first, rows, scales);
    us = rows_rsrc(s.up_scales, first, rows, scales);
  }
};

// SiLU's factor.  bf16: the hardware's 2^x as it is, which makes zeros of results below
// 2^-126 (1 + 2^-126 is 1 all the same), and its reciprocal.
template <typename T>
__device__ __forceinline__ float silu_factor(float v) {
  if constexpr (sizeof(T) == 4) return sigmoid<T>(v);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// Clamped gate and up values and SiLU's factor; NaN passes.
struct Clamped {
  float g, w, s;
  bool off, off_up;
};
template <typename T, bool LIMIT>
__device__ __forceinline__ Clamped clamped(float z, float u, float top) {
  Clamped c;
  c.off = LIMIT && z > top;
  c.off_up = LIMIT && fabsf(u) > top;
  c.g = c.off ? top : z;
  c.w = c.off_up ? copysignf(top, u) : u;
  c.s = silu_factor<T>(c.g);
  return c;
}

// h, and z and u as they are saved.
template <typename T, int KIND>
struct UpOut {
  static constexpr bool sums = false;
  struct Ahead {};
  struct Tile {
    rsrc_t h;
    SavedTile s;
  };
  T *h;
  moe_experts_saved s;
  int N;
  float limit;
  __device__ __forceinline__ Tile begin(const GroupedItem &it, int high) const {
    const int64_t first = (int64_t)it.lo + it.m0;
    const int rows = height(it.n - it.m0, high);
    return Tile{rows_rsrc(h, first, rows, (int64_t)N * sizeof(T)), SavedTile(s, first, rows, N)};
  }
  __device__ __forceinline__ void fetch(const Tile &, Ahead &, int, int) const {}
  template <bool LIMIT>
  __device__ __forceinline__ void glu(float (&v)[8], const float (&u)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Clamped c = clamped<T, LIMIT>(v[j], u[j], limit);
      v[j] = c.g * c.s * c.w;
    }
  }
  __device__ __forceinline__ void put(const Tile &t, const Ahead &, int m, int n, float (&v)[8],
                                      float (&u)[8]) const {
    const uint32_t at = (uint32_t)m * N + n;
    if constexpr (KIND == MOE_SAVE_MXFP8) {
      const uint32_t block = (uint32_t)m * (N / 32) + n / 32;
      keep_piece(v, limit, t.s.z, t.s.zs, at, block, n < N, n % 32 == 0);
      keep_piece(u, limit, t.s.u, t.s.us, at, block, n < N, n % 32 == 0);
    } else if constexpr (KIND == MOE_SAVE_FULL) {
      store_piece<float>(t.s.z, at * 4, v, N - n);
      store_piece<float>(t.s.u, at * 4, u, N - n);
    }
    if (limit > 0.f) glu<true>(v, u);
    else glu<false>(v, u);
    store_piece<T>(t.h, at * sizeof(T), v, N - n);
  }
};

// dz, du and h from dh and the saved z and u.
template <typename T, int KIND>
struct SlopeOut {
  static constexpr bool sums = false, MX = KIND == MOE_SAVE_MXFP8;
  struct Ahead {
    Raw8<float> z, u;          // MXFP8: the codes in the first two words
    uint32_t zs, us;           // and the scales
  };
  struct Tile {
    rsrc_t dz, du, h;
    SavedTile s;
  };
  T *dz, *du, *h;
  moe_experts_saved s;
  int N;
  float limit;
  __device__ __forceinline__ Tile begin(const GroupedItem &it, int high) const {
    const int64_t b = (int64_t)N * sizeof(T), first = (int64_t)it.lo + it.m0;
    const int rows = height(it.n - it.m0, high);
    return Tile{rows_rsrc(dz, first, rows, b), rows_rsrc(du, first, rows, b), rows_rsrc(h, first, rows, b),
                SavedTile(s, first, rows, N)};
  }
  __device__ __forceinline__ void fetch(const Tile &t, Ahead &a, int m, int n) const {
    const uint32_t at = (uint32_t)m * N + n;
    if constexpr (MX) {
      const uint32_t block = n < N ? (uint32_t)m * (N / 32) + n / 32 : kOut;
      const u32x2 z = __builtin_amdgcn_raw_buffer_load_b64(t.s.z, n < N ? at : kOut, 0, 0);
      const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(t.s.u, n < N ? at : kOut, 0, 0);
      a.z.w[0] = z[0]; a.z.w[1] = z[1];
      a.u.w[0] = u[0]; a.u.w[1] = u[1];
      a.zs = __builtin_amdgcn_raw_buffer_load_b8(t.s.zs, block, 0, 0);
      a.us = __builtin_amdgcn_raw_buffer_load_b8(t.s.us, block, 0, 0);
    } else {
      fetch_piece<float>(a.z, t.s.z, at * 4, N - n);
      fetch_piece<float>(a.u, t.s.u, at * 4, N - n);
    }
  }
  // v: dh, then h; z and u, then dz and du
  template <bool LIMIT>
  __device__ __forceinline__ void slopes(float (&v)[8], float (&z)[8], float (&u)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Clamped c = clamped<T, LIMIT>(z[j], u[j], limit);
      const float q = v[j] * c.s;              // dh SiLU's factor
      z[j] = c.off ? 0.f : q * c.w * (1.f + c.g * (1.f - c.s));
      u[j] = c.off_up ? 0.f : q * c.g;
      v[j] = c.g * c.s * c.w;
    }
  }
  __device__ __forceinline__ void put(const Tile &t, const Ahead &a, int m, int n, float (&v)[8],
                                      float (&)[8]) const {
    float z[8], u[8];
    if constexpr (MX) {
      kept<8>(z, {a.z.w[0], a.z.w[1]}, a.zs);
      kept<8>(u, {a.u.w[0], a.u.w[1]}, a.us);
    } else {
      widen8<float>(z, a.z);
      widen8<float>(u, a.u);
    }
    if (limit > 0.f) slopes<true>(v, z, u);
    else slopes<false>(v, z, u);
    const uint32_t off = ((uint32_t)m * N + n) * sizeof(T);
    store_piece<T>(t.dz, off, z, N - n);
    store_piece<T>(t.du, off, u, N - n);
    store_piece<T>(t.h, off, v, N - n);
  }
};

// ---------------------------------------------------------------------------
// A launch's tiles: up to 64 HIGH rows, by the body of their height, 64 NI columns;
// whether its weights are read once (kStream).
template <int H, int N, bool S = false>
struct Shape {
  static constexpr int HIGH = H, NI = N;
  static constexpr bool STREAM = S;
  static constexpr int SLOT = (64 * H + 64 * N) * 64;            // bytes of a stage
  static constexpr int PER_CU = 160 * 1024 / (4 * SLOT);         // workgroups by LDS
};
constexpr int kCus = 256;

// The two operands' copies into the ring: four slots of a stage each, one LDS object
// a slot, B's units first, so that a stage's place and the number of its copies do not
// depend on the height of the tile it belongs to, and the first stages of a tile can
// be asked for while the one before is being stored.
template <typename T, class SH, bool AC, bool BC, bool DUAL>
struct Feed {
  static constexpr int ES = sizeof(T), KB = 64 / ES, HIGH = SH::HIGH, NI = SH::NI;
  static constexpr bool SEGS = !AC && BC;      // two contraction segments (dx)
  static constexpr int AT = 4 * NI * 1024;     // A in a slot
  using OA = Operand<T, AC, 64 * HIGH>;
  using OB = Operand<T, BC, 64 * NI>;
  uint8_t *ring[4];
  int lane, wave, ka;
  uint32_t off_a[HIGH], off_b[NI];
  Cursor ca, cb, cu, ca1, cb1;
  int rest, rest_b, rest1, to_switch, to_switch_b, to_end, to_end_b, nst;

  __device__ __forceinline__ Feed(const GemmOp &g, uint8_t *L0, uint8_t *L1, uint8_t *L2, uint8_t *L3)
      : ring{L0, L1, L2, L3}, lane(threadIdx.x & 63),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) {
    ka = OA::first_k(wave, lane);
#pragma unroll
    for (int q = 0; q < HIGH; ++q) off_a[q] = OA::source(wave + 4 * q, lane, g.a[0].ld);
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      int u = wave + 4 * q;
      if (DUAL && u >= 2 * NI) u -= 2 * NI;
      off_b[q] = OB::source(u, lane, g.b[0].ld);
    }
  }
  // To the first stage of a tile's contraction.
  __device__ __forceinline__ void aim(const GemmOp &g, int m0, int n0) {
    const int st0 = (int)((g.kdim[0] + KB - 1) / KB);
    nst = SEGS && g.segments > 1 ? st0 + (int)((g.kdim[1] + KB - 1) / KB) : st0;
    ca = cursor<T, AC>(g.a[0], m0, 0);
    cb = cursor<T, BC>(g.b[0], n0, 0);
    cu = DUAL ? cursor<T, BC>(g.b_up, n0, 0) : cb;
    ca1 = SEGS ? cursor<T, AC>(g.a[1], m0, 0) : ca;
    cb1 = SEGS ? cursor<T, BC>(g.b[1], n0, 0) : cb;
    to_switch = to_switch_b = SEGS && g.segments > 1 ? st0 : -1;
    rest = rest_b = (int)g.kdim[0];
    rest1 = (int)g.kdim[1];
    to_end = to_end_b = nst;
  }
  template <int VA>
  __device__ __forceinline__ void copy_a(int slot) {
    const rsrc_t r = cursor_rsrc(ca);
    const uint32_t tail = (!AC && ka >= rest) || to_end <= 0 ? kOut : 0u;
#pragma unroll
    for (int q = 0; q < VA; ++q) copy16<0>(r, ring[slot] + AT + (wave + 4 * q) * 1024, off_a[q] | tail);
    ca.p += ca.step; ca.left -= ca.step; rest -= KB; --to_end;
    if constexpr (SEGS) {
      const bool sw = --to_switch == 0;
      ca.p = sw ? ca1.p : ca.p; ca.left = sw ? ca1.left : ca.left; rest = sw ? rest1 : rest;
    }
  }
  __device__ __forceinline__ void copy_b(int slot) {
    const uint32_t tail = (!BC && ka >= rest_b) || to_end_b <= 0 ? kOut : 0u;
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      const int u = wave + 4 * q;
      // units of the second half hold W_up's rows
      const bool up = DUAL && (NI >= 2 ? q >= NI / 2 : u >= 2 * NI);
      copy16<SH::STREAM ? kStream : 0>(cursor_rsrc(up ? cu : cb), ring[slot] + u * 1024, off_b[q] | tail);
    }
    cb.p += cb.step; cb.left -= cb.step; rest_b -= KB; --to_end_b;
    if constexpr (DUAL) { cu.p += cb.step; cu.left -= cb.step; }
    if constexpr (SEGS) {
      const bool sw = --to_switch_b == 0;
      cb.p = sw ? cb1.p : cb.p; cb.left = sw ? cb1.left : cb.left; rest_b = sw ? rest1 : rest_b;
    }
  }
  template <int FIRST, int LAST>
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int p = FIRST; p < LAST; ++p) { copy_a<HIGH>(p); copy_b(p); }
  }
};

constexpr int wait_for(int younger) { return MOE_VMCNT(younger < 63 ? younger : 63); }

// The sums of a tile of MI x 64 rows whose first PRE stages are asked for.  STORES
// stores, those of the tile before, stand between these copies and the next.  vmcnt
// counts in order, so what a stage waits for leaves them out until a stage is needed
// that was asked for after them.  The steps of a stage, and their order: linear.hip.
// Each stage has one way in, from the stage before, so that the compiler can tell which
// copies are under way; where a stage might be skipped it waits for all of them.
template <int MI, int PRE, int STORES, typename T, class SH, bool AC, bool BC, bool DUAL>
__device__ __forceinline__ void sums(Feed<T, SH, AC, BC, DUAL> &f, f32x16 (&acc)[MI][SH::NI]) {
  using F = Feed<T, SH, AC, BC, DUAL>;
  constexpr int NI = SH::NI, ES = sizeof(T);
  // by columns the whole width is copied, whose stride in LDS is one for all heights
  constexpr int VA = AC ? SH::HIGH : MI, VM = VA + NI, VM0 = SH::HIGH + NI;
  const int lane = f.lane, wm = f.wave >> 1, wn = f.wave & 1;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // swiglu: the first half of a wave's column blocks are gate columns, the rest the up
  // columns that go with them
  auto col_block = [&](int j) {
    return DUAL ? (j < NI / 2 ? wn * (NI / 2) + j : NI + wn * (NI / 2) + j - NI / 2) : wn * NI + j;
  };
  u32x4 fa[2][MI], fb[2][NI];
  auto read = [&](int buf, int slot, int s) {
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[buf][j] = F::OB::fragment(f.ring[slot], 0, col_block(j) * 32, s, lane);
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[buf][i] = F::OA::fragment(f.ring[slot], F::AT, (wm * MI + i) * 32, s, lane);
  };
  auto multiply = [&](int buf) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) mma<T>(acc[i][j], fa[buf][i], fb[buf][j]);
  };
  constexpr int kMma = MI * NI * (ES == 2 ? 1 : 4);
  constexpr int kReadsA = MI * (!AC ? 1 : ES == 2 ? 2 : 4);
  constexpr int kReadsB = NI * (!BC ? 1 : ES == 2 ? 2 : 4);

  f.template start<PRE, 3>();
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(wait_for(2 * VM0 + STORES));
  __builtin_amdgcn_s_barrier();
  read(0, 0, 0);
  auto stage = [&](int p, auto early) {
    __builtin_amdgcn_sched_barrier(0);
    read(1, p, 1);
    f.template copy_a<VA>((p + 3) % 4);
    multiply(0);
    interleave<0, kMma, kReadsA + kReadsB, VA>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_for(VM + VA + (early ? STORES : 0)) & ~(15 << 8));   // and lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(0, (p + 1) % 4, 0);
    f.copy_b((p + 3) % 4);
    multiply(1);
    interleave<0, kMma, kReadsA + kReadsB, NI>();
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::false_type later{};
  constexpr std::bool_constant<(STORES > 0)> early{};
  int left = f.nst;
  if (STORES > 0 && left >= 4) {
    stage(0, early);
    stage(1, early);
    stage(2, later);
    stage(3, later);
    left -= 4;
  }
  for (; left >= 4; left -= 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) stage(p, later);
  }
  if (left > 0) {
    stage(0, later);
    if (left > 1) {
      stage(1, later);
      if (left > 2) stage(2, later);
    }
  }
  // the copies past the end have landed, and every wave is done with the ring
  __builtin_amdgcn_s_waitcnt(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// A workgroup's tiles, one after another: next(it) finds its next one.
template <typename T, class SH, bool AC, bool BC, bool DUAL, class OUT, class NEXT, class AIM>
__device__ __forceinline__ void walk(const GemmOp &g, const OUT &out, NEXT next, AIM aim) {
  __shared__ __attribute__((aligned(1024))) uint8_t L0[SH::SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t L1[SH::SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t L2[SH::SLOT];
  __shared__ __attribute__((aligned(1024))) uint8_t L3[SH::SLOT];
  constexpr int NI = SH::NI, NJ = DUAL ? NI / 2 : NI, HIGH = SH::HIGH;
  // The end of a tile goes through LDS, so that a store's lanes write whole lines
  // (straight from the accumulators, 32 bytes a row and store, 16384 rows of 64 experts
  // took 271 us for dW of 2048 -> 2 x 1024, through LDS 245: the L2 takes a request a
  // piece).  Of the largest tiles through memory of its own beside the ring, so that
  // the next one's first stages can be asked for before; of others the ring itself,
  // where that would cost a CU a workgroup.
  constexpr int PASS = NI >= 2 ? 2 : 1;        // blocks of a wave there at a time
  constexpr int BYTES = PASS * 1024 * (OUT::sums ? (int)sizeof(T) : 4);
  constexpr bool OWN = SH::PER_CU == 1;
  constexpr int PRE = OWN ? 3 : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t ends[OWN ? 4 * BYTES : 16];
  // Stores of a tile's end where they stand after copies, the same for every height and
  // before the first tile.
  constexpr int STORES = OWN && OUT::sums ? HIGH * NI * (int)sizeof(T) : 0;
  auto no_stores = [](int n) {
    const rsrc_t none = __builtin_amdgcn_make_buffer_rsrc(nullptr, 0, 0, 0x00027000);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, none, kOut, 0, 0);
      asm volatile("" ::: "memory");           // each one its own: they are counted
    }
  };
  GroupedItem first;
  if (!next(&first)) return;
  Feed<T, SH, AC, BC, DUAL> f(g, L0, L1, L2, L3);
  const int lane = f.lane, wave = f.wave, wm = wave >> 1, wn = wave & 1;
  aim(f, first, first.nt * 64 * NJ);
  f.template start<0, PRE>();
  __builtin_amdgcn_sched_barrier(0);
  no_stores(STORES);
  __builtin_amdgcn_sched_barrier(0);
  walk_tiles<HIGH>(first, [&](auto height, const GroupedItem &it, GroupedItem &nx) {
    constexpr int MI = decltype(height)::value;
    f32x16 acc[MI][NI];
    sums<MI, PRE, STORES>(f, acc);
    const bool more = next(&nx);
    const int n0 = it.nt * 64 * NJ;
    // The next tile's first stages; without one copies that read nothing, so that their
    // number is known where a load's wait counts them.
    auto ask = [&]() {
      if (more) aim(f, nx, nx.nt * 64 * NJ);
      else f.to_end = f.to_end_b = 0;
      f.template start<0, PRE>();
    };
    const auto t = out.begin(it, MI * 64);
    constexpr bool TWO = 2 * BYTES <= SH::SLOT;        // waves to a slot
    static_assert(BYTES <= SH::SLOT, "they fit");
    uint8_t *stage = OWN ? ends + wave * BYTES
                     : TWO ? (wave < 2 ? L0 : L1) + (wave & 1) * BYTES
                           : (wave == 0 ? L0 : wave == 1 ? L1 : wave == 2 ? L2 : L3);
    // 16-byte chunk c of row r lies at chunk c ^ (r % 8) (of four to a row, r % 4): a
    // column of chunks, which lanes write together, and a row of them, which they read,
    // take all banks
    constexpr int CHUNKS = BYTES / 32 / 16, SWAP = CHUNKS < 8 ? CHUNKS - 1 : 7;
    auto chunk = [&](int r, int c) { return stage + r * (BYTES / 32) + ((c ^ (r & SWAP)) << 4); };
    if constexpr (OUT::sums) {
      constexpr int PC = CHUNKS;               // pieces of a row
      constexpr int ROWS = 64 / PC;            // rows that the wave takes at once
      if (OWN) ask();
      __builtin_amdgcn_sched_barrier(0);       // sums() counts these copies before the stores
      const int r0 = lane / PC, pc = lane % PC;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; j += PASS) {
#pragma unroll
          for (int k = 0; k < PASS; ++k) {
            f32x16 a = acc[i][j + k];
            asm volatile("" : "+v"(a));        // rounded here, not all blocks ahead
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (sizeof(T) == 2) {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                *(bf16x4 *)(chunk(lane & 31, 4 * k + e) + 8 * (lane >> 5)) =
                    bf16x4{(bf16)a[4 * e], (bf16)a[4 * e + 1], (bf16)a[4 * e + 2], (bf16)a[4 * e + 3]};
              } else {
                *(f32x4 *)chunk(lane & 31, 8 * k + 2 * e + (lane >> 5)) =
                    f32x4{a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]};
              }
            }
          }
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int q = 0; q < 32 / ROWS; ++q)
            out.put(t, (wm * MI + i) * 32 + r0 + q * ROWS,
                    n0 + (wn * NI + j) * 32 + pc * (16 / (int)sizeof(T)),
                    *(const u32x4 *)chunk(r0 + q * ROWS, pc));
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_sched_barrier(0);   // a pass's registers at a time
        }
      if (STORES > 0) no_stores((HIGH - MI) * NI * (int)sizeof(T));
    } else {
      // PASS blocks at a time (swiglu: one of the gate and the up one that goes with it)
      // through the wave's part of LDS, then a piece of eight columns a lane.  The
      // blocks' and the pieces' loops stay loops: unrolled, the code of these endings
      // would not stay in the instruction cache.  What the next piece reads is asked for
      // before this one's stores.
      constexpr int COLS = DUAL ? 1 : PASS;    // blocks of output columns a pass
      constexpr int PC = COLS * 4;             // pieces of a row
      constexpr int PPL = 32 * PC / 64;        // pieces of a lane and pass
      constexpr int ROWS = 64 / PC;            // rows that the wave takes at once
      constexpr int PER_ROW = NJ / COLS;       // passes in 32 rows
      static_assert(NJ % COLS == 0, "passes divide the columns");
      const int r0 = lane / PC, pc = lane % PC;
      const int m0 = wm * MI * 32 + r0, c0 = n0 + wn * NJ * 32 + pc * 8;
      typename OUT::Ahead ahead, now;
      out.fetch(t, ahead, m0, c0);
      if (OWN) ask();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll 1
      for (int b = 0; b < MI * PER_ROW; ++b) {
#pragma unroll
        for (int k = 0; k < MI * PER_ROW; ++k)
          if (k == b) {                        // uniform; the accumulators keep their registers
#pragma unroll
            for (int j = 0; j < PASS; ++j) {
              const f32x16 &a = acc[k / PER_ROW][DUAL ? k % PER_ROW + j * NJ : k % PER_ROW * PASS + j];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *(f32x4 *)chunk(lane & 31, j * 8 + 2 * e + (lane >> 5)) =
                    f32x4{a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]};
            }
          }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 2
        for (int q = 0; q < PPL; ++q) {
          auto at = [&](int pass, int piece, int *m, int *n) {
            *m = m0 + pass / PER_ROW * 32 + piece * ROWS;
            *n = c0 + pass % PER_ROW * COLS * 32;
          };
          int m, n, m1, n1;
          at(b, q, &m, &n);
          at(q + 1 < PPL ? b : b + 1, q + 1 < PPL ? q + 1 : 0, &m1, &n1);
          now = ahead;
          out.fetch(t, ahead, m1, n1);         // past the last: rows that are not there
          const int r = r0 + q * ROWS;
          float v[8], u[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f32x4 x = *(const f32x4 *)chunk(r, 2 * pc + h);
            f32x4 y = x;
            if constexpr (DUAL) y = *(const f32x4 *)chunk(r, 8 + 2 * pc + h);
#pragma unroll
            for (int j = 0; j < 4; ++j) { v[4 * h + j] = x[j]; u[4 * h + j] = y[j]; }
          }
          out.put(t, now, m, n, v, u);
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
    if constexpr (!OWN) {
      // this part of the ring is the next tile's again
      __builtin_amdgcn_s_waitcnt(MOE_VMCNT(63) & ~(15 << 8));
      __builtin_amdgcn_s_barrier();
      ask();
    }
    __builtin_amdgcn_sched_barrier(0);
    return more;
  });
  __builtin_amdgcn_s_waitcnt(0);               // no copy into LDS outlives the workgroup
}

// Products over rows.  Items go expert by expert, a column tile's row tiles together;
// each XCD takes a contiguous run of them and its workgroups go through it side by
// side: the rows of an expert and the weights of a column tile are then read through
// one L2.  (Contiguous shares for the workgroups, all of one size, spread an XCD over
// eight experts at a time: 16384 rows of 64 experts, 2048 -> 2 x 1024, 267 us where
// this order took 217.)
template <typename T, class SH, bool BC, bool DUAL, class OUT>
__device__ __forceinline__ void rows_product(const GroupedOp &q, const OUT &out) {
  const auto line = line_of<int>(q.E, [&](int e) { return tiles_of<SH::HIGH>(span_of(q, e).n); });
  const int nt = q.g.n_tiles, items = line.total() * nt, per = (items + 7) / 8;
  const int run = (int)(blockIdx.x & 7) * per, mine = items - run < per ? items - run : per;
  // Tiles of a last round that leave half of the XCD's places free are cut lower, into
  // `cut` parts each (64 experts, 2048 -> 2 x 1024, 16384 rows 249 us, cut 238; 32768
  // rows 380 and 357; dh and dx by 0 to 5 %).
  const int places = (int)(gridDim.x >> 3);
  const int last = mine > 0 ? mine % places : 0, whole = mine - last;
  const int cut = SH::HIGH >= 4 && last * 4 <= places ? 4 : SH::HIGH >= 2 && last * 2 <= places ? 2 : 1;
  int slot = (int)(blockIdx.x >> 3) - places;
  auto next = [&](GroupedItem *it) {
    for (;;) {
      slot += places;
      const int behind = slot - whole;
      if (behind >= last * cut) return false;
      const int item = run + (behind < 0 ? slot : whole + behind / cut);
      int start;
      it->e = line.at(item / nt, &start);
      const Span s = span_of(q, it->e);
      it->lo = __builtin_amdgcn_readfirstlane(s.lo);
      it->n = __builtin_amdgcn_readfirstlane(s.n);
      const int high = tiles_of<SH::HIGH>(it->n), local = item - start * nt;
      it->nt = local / high;
      it->half = 0;
      height_of((it->n + 63) / 64, high, local - it->nt * high, it);
      if (behind >= 0 && cut > 1) {
        const int m0 = it->m0;
        height_of(it->blocks, cut, behind % cut, it);
        it->m0 += m0;
        if (it->blocks == 0) continue;
      }
      return true;
    }
  };
  walk<T, SH, false, BC, DUAL>(q.g, out, next, [&](auto &f, const GroupedItem &it, int n0) {
    GemmOp g = q.g;
    move<T>(g.a[0], it);
    move<T>(g.a[1], it);
    g.b[0].p = (const uint8_t *)g.b[0].p + it.e * q.b_expert;
    g.b[1].p = (const uint8_t *)g.b[1].p + it.e * q.b_expert;
    g.b_up.p = (const uint8_t *)g.b_up.p + it.e * q.b_expert;
    f.aim(g, it.m0, n0);
  });
}

template <typename T, class SH, int KIND>
__global__ __launch_bounds__(256, SH::PER_CU) void up_kernel(const GroupedOp q, const UpOut<T, KIND> o) {
  rows_product<T, SH, false, true>(q, o);
}
template <typename T, class SH>
__global__ __launch_bounds__(256, SH::PER_CU) void down_kernel(const GroupedOp q, const SumsOut<T> o) {
  rows_product<T, SH, false, false>(q, o);
}
template <typename T, class SH, int KIND>
__global__ __launch_bounds__(256, SH::PER_CU) void dh_kernel(const GroupedOp q, const SlopeOut<T, KIND> o) {
  rows_product<T, SH, true, false>(q, o);
}
template <typename T, class SH>
__global__ __launch_bounds__(256, SH::PER_CU) void dx_kernel(const GroupedOp q, const SumsOut<T> o) {
  rows_product<T, SH, true, false>(q, o);
}

// Weight gradients: every expert has the same tiles, those of an expert without rows
// are zeros.  An XCD takes the tiles of a range of experts, ranges of equal cost
// (stages, and kTileStages for what a tile costs besides), and its workgroups go
// through them side by side: the rows that they read lie in its L2.
constexpr int kTileStages = 8;
template <typename T, class SH>
__global__ __launch_bounds__(256, SH::PER_CU) void dw_kernel(const GroupedOp q, const SumsOut<T> o) {
  constexpr int KB = 64 / sizeof(T);
  const int tiles = (int)q.g.m_tiles * q.g.n_tiles, per_half = (int)q.g.m_tiles / q.g.halves;
  auto cost = [&](int e) { return (span_of(q, e).n + KB - 1) / KB + kTileStages; };
  const auto line = line_of<int64_t>(q.E, [&](int e) { return (int64_t)cost(e) * tiles; });
  auto first_of = [&](int xcd) {
    const int64_t pos = line.total() / 8 * xcd;
    int64_t start;
    const int e = line.at(pos, &start);
    return e * tiles + (int)((pos - start) / __builtin_amdgcn_readfirstlane(cost(e)));
  };
  const int xcd = (int)(blockIdx.x & 7), places = (int)(gridDim.x >> 3);
  const int last = xcd == 7 ? tiles * q.E : first_of(xcd + 1);
  int item = first_of(xcd) + (int)(blockIdx.x >> 3) - places;
  auto next = [&](GroupedItem *it) {
    item += places;
    if (item >= last) return false;
    it->e = item / tiles;
    const int local = item - it->e * tiles;
    int mt = local / q.g.n_tiles;
    it->nt = local - mt * q.g.n_tiles;
    it->half = mt >= per_half ? 1 : 0;
    mt -= it->half * per_half;
    height_of((int)((q.g.M + 63) / 64), per_half, mt, it);
    const Span s = span_of(q, it->e);
    it->lo = __builtin_amdgcn_readfirstlane(s.lo);
    it->n = __builtin_amdgcn_readfirstlane(s.n);
    return true;
  };
  walk<T, SH, true, true, false>(q.g, o, next, [&](auto &f, const GroupedItem &it, int n0) {
    GemmOp g = q.g;
    if (it.half) g.a[0] = g.a_up;
    move<T>(g.a[0], it);
    move<T>(g.b[0], it);
    g.kdim[0] = it.n;
    f.aim(g, it.m0, n0);
  });
}

// ---------------------------------------------------------------------------
// The most 64-row blocks of `rows` rows of E experts.
int64_t most_blocks(int64_t rows, int E) { return rows / 64 + (rows < E ? rows : E); }

GroupedOp grouped_op(const ExpertsArgs &a, int N) {
  GroupedOp q = {};
  q.offsets = a.offsets;
  q.rows = a.rows;
  q.E = a.E;
  q.g.segments = 1;
  q.g.parts = 1;
  q.g.halves = 1;
  q.g.e.N = N;
  return q;
}

// Workgroups: what the GPU holds, or fewer where there is less to do.
template <class SH>
dim3 held_grid(int64_t items) {
  const int64_t most = kCus * SH::PER_CU, n = (items + 7) / 8 * 8;
  return dim3((unsigned)(n < most ? n : most));
}

// Sets a product's column tiles; its workgroups.
template <class SH>
dim3 rows_grid(GroupedOp &q, bool dual) {
  const int to = dual ? 32 * SH::NI : 64 * SH::NI;
  q.g.n_tiles = (q.g.e.N + to - 1) / to;
  return held_grid<SH>(most_blocks(q.rows, q.E) * q.g.n_tiles);
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
  // Tiles are counted in 31 bits, by workgroups that step past the last; the smallest are
  // the most.  Offsets that are not ascending can give every second expert all rows, and
  // where experts follow one another each can have a block that is not whole.
  const int64_t down = (a.d + 63) / 64, up = (a.I + 31) / 32, most = INT32_MAX - 1024;
  const int64_t by_rows = ((a.E + 1) / 2 * (a.rows / 64) + a.E) * (down > up ? down : up);
  const int64_t by_expert =
      backward ? 2 * (int64_t)a.E * ((a.d + 63) / 64) * ((a.I + 63) / 64) : 0;
  return by_rows < most && by_expert < most;
}

namespace {

// Tile shape of a product: the largest tiles of which there are about as many as CUs,
// counting for a product over rows experts with the mean's rows and half a tile each
// left over.  bf16, microseconds, each shape forced on 20 problems (120 products), 256 x
// 256 against 128 x 128:
//   256 tiles: 4096 rows of one expert, 4096 -> 2 x 2048, up 126 and 188, down 65 and 95, dx
//   112 and 159; 240: 8192 of 16, 1024 -> 2 x 768, up 46 and 49; 192: 4096 of 16, 2048 -> 2 x
//   1024, up 64 and 61, dx 52 and 55; 144: 8192 of 8, 2048 -> 2 x 1024, dh 67 and 56
// and 128 x 128 against 64 x 64:
//   288 tiles: 4096 of 8, 2048 -> 2 x 1024, dh 39 and 45; 272: 4096 of 4, 1024 -> 2 x 1024,
//   down 21 and 26; 160: 8192 of 33, 512 -> 2 x 256, dh 16.0 and 14.9, but 2048 of 8, 1024 ->
//   2 x 1024, down 13.3 and 16.3; 92: 2000 of 16, 512 -> 2 x 512, down 7.9 and 7.5
// Products over rows lose 3 % on the mean to the best shape, 26 % at most (dx of those 2048
// rows: 25.8, 128 x 128 20.5).  Weight gradients lose 8 % and up to 48 %: the endings of 256 x
// 256 weigh on a few hundred rows an expert, where 128 x 128 is the faster to some 500 tiles
// (256 tiles: dWd of 4096 of 8, 2048 -> 2 x 1024, 36 and 26; but dWg and dWu of one expert's 4096
// rows, 4096 -> 2 x 2048, 109 and 159; 512: dWg and dWu of the former 50 and 47).
// up has two matrices in a tile, 64 x 128 at least.  fp32 has 64 x 64 alone: 2048 rows of 16
// experts, 1024 -> 2 x 512, all six 315, with 128 x 128 363, where the matrix cores' rate
// would allow 128: the contractions are short, and nothing runs beside the one or two tiles'
// first copies and endings.
//
// The products forward of a few rows an expert are a stream of weights, and take 64 x 256,
// of which two workgroups fit a CU.  up and down, 64 x 256 against 256 x 256:
//    2 rows an expert  32 experts, 7168 -> 2 x 2048  296, 134 and 312, 137
//   16                                               360, 189 and 366, 196
//   20                                               360, 189 and 365, 194
//   24                                               467, 189 and 374, 195
//   16                 64 experts, 2048 -> 2 x 1024  137, 59 and 144, 61
//   20                                               156, 68 and 141, 60
//   24                 48 experts, 5120 -> 2 x 1536  352, 161 and 371, 168
//   32                                               356, 184 and 376, 169
// (from where the fullest experts have more than 64 rows they take a second tile).
//
// Weights by columns are streamed where an expert has two row tiles of the largest on
// the mean, or fewer.  dh and dx streamed, and not:
//   rows an expert   64 experts, 2048 -> 2 x 1024    48 experts, 5120 -> 2 x 1536
//        64           77, 110 and  88, 120           212, 323 and 229, 337
//       128          106, 142 and 119, 146           247, 372 and 252, 384
//       256          141, 175 and 135, 171           324, 519 and 322, 484
//       512          256, 305 and 229, 285           536, 861 and 501, 777
//       640          293, 376 and 282, 373           673, 1042 and 560, 918
//      1024          422, 536 and 377, 501          1010, 1522 and 842, 1354
// so of one row tile it gains up to some 200 rows an expert, and of two it loses.
struct Pick {
  int high, ni;
  bool stream;
};
Pick pick(const ExpertsArgs &a, int product) {
  const bool rows_product = product <= MOE_EXPERTS_DX, dw = product == MOE_EXPERTS_DW;
  const int64_t d = a.d, I = a.I, experts = a.rows < a.E ? a.rows : a.E;
  const int64_t cols = product == MOE_EXPERTS_UP ? 2 * I
                       : product == MOE_EXPERTS_DOWN || product == MOE_EXPERTS_DX || dw ? d : I;
  auto tiles = [&](int high, int wide) {
    const int64_t across = (cols + 64 * wide - 1) / (64 * wide);
    if (!rows_product) return a.E * (((dw ? 2 * I : d) + 64 * high - 1) / (64 * high)) * across;
    const int64_t by_rows = a.rows / (64 * high) + experts / 2;
    return (by_rows > experts ? by_rows : experts) * across;
  };
  if (a.dtype == MOE_DTYPE_BF16) {
    if (product <= MOE_EXPERTS_DOWN && a.rows <= 16 * (int64_t)a.E && tiles(1, 4) >= 200)
      return {1, 4, false};
    if (tiles(4, 4) >= 200) {
      const bool by_columns = product == MOE_EXPERTS_DH || product == MOE_EXPERTS_DX;
      return {4, 4, by_columns && a.rows <= 512 * (int64_t)a.E};
    }
    if (tiles(2, 2) >= 256) return {2, 2, false};
  }
  return {1, product == MOE_EXPERTS_UP ? 2 : 1, false};
}

// Calls f with the shape that is picked.
template <typename T, int PRODUCT, class F>
hipError_t with_shape(const ExpertsArgs &a, F f) {
  const Pick t = pick(a, PRODUCT);
  if constexpr (sizeof(T) == 2) {
    if constexpr (PRODUCT == MOE_EXPERTS_DH || PRODUCT == MOE_EXPERTS_DX)
      if (t.stream) return f(Shape<4, 4, true>{});
    if constexpr (PRODUCT <= MOE_EXPERTS_DOWN)
      if (t.high == 1 && t.ni == 4) return f(Shape<1, 4>{});
    if (t.high == 4) return f(Shape<4, 4>{});
    if (t.high == 2) return f(Shape<2, 2>{});
  }
  return f(Shape<1, PRODUCT == MOE_EXPERTS_UP ? 2 : 1>{});
}

// Calls f with the saved kind as a constant.
template <class F>
hipError_t with_kind(int kind, F f) {
  if (kind == MOE_SAVE_MXFP8) return f(std::integral_constant<int, MOE_SAVE_MXFP8>{});
  if (kind == MOE_SAVE_FULL) return f(std::integral_constant<int, MOE_SAVE_FULL>{});
  return f(std::integral_constant<int, MOE_SAVE_NONE>{});
}

template <typename T>
hipError_t run_up(const ExpertsArgs &a, T *h, hipStream_t s) {
  GroupedOp q = grouped_op(a, a.I);
  q.g.a[0] = {a.x, a.d, a.rows, a.d};
  q.g.b[0] = {a.w_gate, a.d, a.I, a.d};
  q.g.b_up = {a.w_up, a.d, a.I, a.d};
  q.b_expert = (int64_t)a.I * a.d * sizeof(T);
  q.g.kdim[0] = a.d;
  return with_shape<T, MOE_EXPERTS_UP>(a, [&](auto sh) {
    using SH = decltype(sh);
    const dim3 grid = rows_grid<SH>(q, true);
    return with_kind(a.saved.kind, [&](auto kind) {
      const UpOut<T, kind> o = {h, a.saved, a.I, a.limit};
      hipLaunchKernelGGL((up_kernel<T, SH, kind>), grid, dim3(256), 0, s, q, o);
      return hipGetLastError();
    });
  });
}

template <typename T>
hipError_t run_down(const ExpertsArgs &a, const T *h, hipStream_t s) {
  GroupedOp q = grouped_op(a, a.d);
  q.g.a[0] = {h, a.I, a.rows, a.I};
  q.g.b[0] = {a.w_down, a.I, a.d, a.I};
  q.b_expert = (int64_t)a.I * a.d * sizeof(T);
  q.g.kdim[0] = a.I;
  const SumsOut<T> o = {(T *)a.y, nullptr, a.d, 0};
  return with_shape<T, MOE_EXPERTS_DOWN>(a, [&](auto sh) {
    using SH = decltype(sh);
    const dim3 grid = rows_grid<SH>(q, false);
    hipLaunchKernelGGL((down_kernel<T, SH>), grid, dim3(256), 0, s, q, o);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t run_dh(const ExpertsArgs &a, T *dz, T *du, T *h, hipStream_t s) {
  GroupedOp q = grouped_op(a, a.I);
  q.g.a[0] = {a.dy, a.d, a.rows, a.d};
  q.g.b[0] = {a.w_down, a.I, a.d, a.I};
  q.b_expert = (int64_t)a.I * a.d * sizeof(T);
  q.g.kdim[0] = a.d;
  return with_shape<T, MOE_EXPERTS_DH>(a, [&](auto sh) {
    using SH = decltype(sh);
    const dim3 grid = rows_grid<SH>(q, false);
    if (a.saved.kind == MOE_SAVE_MXFP8) {
      const SlopeOut<T, MOE_SAVE_MXFP8> o = {dz, du, h, a.saved, a.I, a.limit};
      hipLaunchKernelGGL((dh_kernel<T, SH, MOE_SAVE_MXFP8>), grid, dim3(256), 0, s, q, o);
    } else {
      const SlopeOut<T, MOE_SAVE_FULL> o = {dz, du, h, a.saved, a.I, a.limit};
      hipLaunchKernelGGL((dh_kernel<T, SH, MOE_SAVE_FULL>), grid, dim3(256), 0, s, q, o);
    }
    return hipGetLastError();
  });
}

template <typename T>
hipError_t run_dx(const ExpertsArgs &a, const T *dz, const T *du, hipStream_t s) {
  GroupedOp q = grouped_op(a, a.d);
  q.g.a[0] = {dz, a.I, a.rows, a.I};
  q.g.a[1] = {du, a.I, a.rows, a.I};
  q.g.b[0] = {a.w_gate, a.d, a.I, a.d};
  q.g.b[1] = {a.w_up, a.d, a.I, a.d};
  q.b_expert = (int64_t)a.I * a.d * sizeof(T);
  q.g.kdim[0] = q.g.kdim[1] = a.I;
  q.g.segments = 2;
  const SumsOut<T> o = {(T *)a.dx, nullptr, a.d, 0};
  return with_shape<T, MOE_EXPERTS_DX>(a, [&](auto sh) {
    using SH = decltype(sh);
    const dim3 grid = rows_grid<SH>(q, false);
    hipLaunchKernelGGL((dx_kernel<T, SH>), grid, dim3(256), 0, s, q, o);
    return hipGetLastError();
  });
}

// A weight gradient [N, K] of every expert: columns of A (and A_up), columns of B.
template <typename T, bool DOWN>
hipError_t run_dw(const ExpertsArgs &a, const void *A, const void *A_up, int N, const void *B, int K,
                  void *dw, void *dw_up, hipStream_t s) {
  GroupedOp q = grouped_op(a, K);
  q.g.a[0] = {A, N, a.rows, N};
  q.g.a_up = {A_up, N, a.rows, N};
  q.g.b[0] = {B, K, a.rows, K};
  q.g.M = N;
  q.g.halves = A_up ? 2 : 1;
  const SumsOut<T> o = {(T *)dw, (T *)dw_up, K, N};
  auto run = [&](auto sh) {
    using SH = decltype(sh);
    q.g.m_tiles = (N + 64 * SH::HIGH - 1) / (64 * SH::HIGH) * q.g.halves;
    q.g.n_tiles = (K + 64 * SH::NI - 1) / (64 * SH::NI);
    const dim3 grid = held_grid<SH>(q.g.m_tiles * q.g.n_tiles * a.E);
    hipLaunchKernelGGL((dw_kernel<T, SH>), grid, dim3(256), 0, s, q, o);
    return hipGetLastError();
  };
  // one of gate and up alone takes the tiles of both, and comes out the same
  return DOWN ? with_shape<T, MOE_EXPERTS_DW_DOWN>(a, run) : with_shape<T, MOE_EXPERTS_DW>(a, run);
}

template <typename T>
hipError_t run_forward(const ExpertsArgs &a, char *ws, hipStream_t s) {
  T *h = (T *)(ws + experts_space(a.rows, a.I, a.dtype, false).h);
  const hipError_t err = run_up<T>(a, h, s);
  return err != hipSuccess ? err : run_down<T>(a, h, s);
}

template <typename T>
hipError_t run_backward(const ExpertsArgs &a, char *ws, hipStream_t s) {
  const ExpertsSpace L = experts_space(a.rows, a.I, a.dtype, true);
  T *h = (T *)(ws + L.h), *dz = (T *)(ws + L.dz), *du = (T *)(ws + L.du);
  hipError_t err;
  if (a.rows > 0 && (err = run_dh<T>(a, dz, du, h, s)) != hipSuccess) return err;
  if (a.dw_down &&
      (err = run_dw<T, true>(a, a.dy, nullptr, a.d, h, a.I, a.dw_down, nullptr, s)) != hipSuccess)
    return err;
  if (a.dw_gate || a.dw_up) {
    // both in one launch, or the one that is wanted
    const bool both = a.dw_gate && a.dw_up;
    if ((err = run_dw<T, false>(a, a.dw_gate ? dz : du, both ? du : nullptr, a.I, a.x, a.d,
                         a.dw_gate ? a.dw_gate : a.dw_up, a.dw_up, s)) != hipSuccess)
      return err;
  }
  if (a.dx && a.rows > 0) return run_dx<T>(a, dz, du, s);
  return hipSuccess;
}

}  // namespace

moe_experts_path_info experts_path(const ExpertsArgs &a, int product) {
  const Pick t = pick(a, product);
  return {64 * t.high, 64 * t.ni, t.stream};
}

hipError_t launch_experts(const ExpertsArgs &a, char *ws, hipStream_t s) {
  return a.dtype == MOE_DTYPE_F32 ? run_forward<float>(a, ws, s) : run_forward<bf16>(a, ws, s);
}

hipError_t launch_experts_backward(const ExpertsArgs &a, char *ws, hipStream_t s) {
  return a.dtype == MOE_DTYPE_F32 ? run_backward<float>(a, ws, s) : run_backward<bf16>(a, ws, s);
}

}  // namespace moe
