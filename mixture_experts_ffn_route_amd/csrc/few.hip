// The MoE layer for a few tokens (1 .. 16): moe_forward_few.
//
//   y[t] = sum_j w[t,j] FFN_{idx[t,j]}(x[t]) + FFN_shared(x[t])
//
// At these sizes the layer is a stream of the chosen experts' weights: every
// weight is used by one or two tokens, so the time is (bytes of the distinct
// chosen experts) / (HBM rate) plus launches and the waits between dependent
// steps.  Four or five launches, no permutation:
//   few_scores   gate logits (a small gate's: few_plan); MXFP8 codes of x
//   few_plan     one workgroup selects the experts of every token and lists the
//                distinct ones ("slots"); meanwhile the others stream the shared
//                expert's gate|up, which needs x alone
//   few_up       H = SwiGLU of every (slot, token)
//   few_down     w (H W_down^T) of every (slot, token), and the shared rows
//   few_combine  the sum over a token's experts
//
// The token is the MFMA row: a product covers 16 rows x 16 weight columns, row
// t is token t for every expert.  Rows of tokens that did not choose the expert
// are read as zeros and not stored.  The padded rows cost MFMA issue slots
// only, which a weight stream has to spare (a 1 KB weight fragment arrives per
// ~100 cycles and CU at the HBM rate; its MFMA takes 16).
//
// What bounds a weight stream here, from a read-only kernel on 700 MB (TB/s):
// 16 rows x 64 bytes per load, the MFMA operand order of row-layout weights,
// 4.5 - 5.5; 8 rows x 128 bytes, whole cache lines, 6.7 - 7.0; contiguous 1 KB
// (tiled layout) the same.  So weights are copied line-wise into a wave's own
// part of LDS (asynchronous 16-byte copies, no barrier) and read back in
// operand order.  Every vector memory instruction also costs its 16 cycles of
// the CU's address and return path, also one whose lanes are all out of range:
// a wave takes 64 weight rows at a time, so that the token rows (16-byte loads
// from L2) are few next to the weights, and issues no load past its share.
//
// Measured (microseconds of the launches, row-layout weights): V4.1-Flash-shaped
// FP4 experts on bf16 activations, one token (151 MB of weights): scores 4, plan
// 11, up 17, down 14, combine 4; five tokens (532 MB): 5, 13, 61 (5.3 TB/s), 37,
// 5; 16 tokens on MXFP8 activations (1.43 GB): 5, 20, 141 (6.5 TB/s), 88, 5.
// V3-shaped bf16 experts, one token (796 MB): 4, 13, 71 (6.6 TB/s), 42, 4.
// What is left over the weights' time is each launch's start (a first load
// takes 2 - 3 us), the shared expert's gate|up on one workgroup per 16 columns (at
// one token that stream, 34 KB a microsecond and CU, is the plan launch's time, at
// 16 the routing is), and at one token the CUs that up, down and combine leave idle.

#include <climits>

#include "gemm.h"
#include "few.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kRows = MOE_FEW_MAX_TOKENS;      // MFMA rows = tokens
constexpr int kLogitParts = 8;
constexpr uint32_t kOut = 0x80000000u;         // an offset no resource here reaches: reads 0

// Weight formats of a product.
enum { F_F32, F_BF16, F_FP4, F_MX4, F_MX8 };

// Inputs of one stage, the unit of a wave's load ring: 128 bytes of a weight
// row (fp32 layers, which load straight to registers: 64).
template <int F> constexpr int stage_inputs() {
  return F == F_F32 ? 16 : F == F_BF16 ? 64 : F == F_MX8 ? 128 : 256;
}
// Bytes of a weight row of K inputs.
template <int F> __device__ __forceinline__ int64_t row_bytes(int64_t K) {
  return F == F_F32 ? 4 * K : F == F_BF16 ? 2 * K : F == F_MX8 ? K : K / 2;
}

__device__ __forceinline__ rsrc_t resource(const void *p, int64_t bytes) {
  const uint32_t n = bytes < 0 ? 0 : bytes < (int64_t)kOut ? (uint32_t)bytes : kOut;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, n, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
}
__device__ __forceinline__ uint32_t load4(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
__device__ __forceinline__ uint32_t load1(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
}

// ---------------------------------------------------------------------------
// Weights.  A wave's tile is 2 x 16 NB rows: NB row blocks of each of two
// sources (gate and up, or the two halves of 32 NB rows of W_down).
struct WSrc {
  rsrc_t r, rs;                                // the rows, their scales
};
// Rows n0 .. n0 + rows - 1 of an [N, K] matrix.
template <int F>
__device__ __forceinline__ WSrc w_source(const void *mat, const uint8_t *sc, int N, int K, int n0,
                                         int rows) {
  WSrc w;
  const int have = N - n0 < rows ? N - n0 : rows;
  const int64_t rb = row_bytes<F>(K);
  w.r = resource((const uint8_t *)mat + n0 * rb, have * rb);
  if constexpr (F == F_MX8)
    w.rs = resource(sc + (int64_t)(n0 / 128) * (K / 128), have > 0 ? K / 128 : 0);
  else if constexpr (F == F_FP4 || F == F_MX4)
    w.rs = resource(sc + (int64_t)n0 * (K / 32), (int64_t)have * (K / 32));
  else
    w.rs = w.r;
  return w;
}

// Stage st of a source's 16 NB rows, copied to `lds` (2 KB a row block).
//   rows layout: unit u is 8 rows x 128 bytes, row r's 16-byte piece c at
//     position c ^ (r % 8): the operand reads below then take distinct banks
//     (address bits 4..8, bit 10 folded into bit 8, within a half-wave)
//   tiled layout: the row block's 2 KB as they lie
template <int F, bool TILED, int NB>
__device__ __forceinline__ void copy_stage(const WSrc &w, int K, int lane, int st, uint8_t *lds) {
  const uint32_t rb = (uint32_t)row_bytes<F>(K);
#pragma unroll
  for (int u = 0; u < 2 * NB; ++u) {
    uint32_t off;
    if constexpr (TILED) {
      // row block u / 2, its 1 KB half u % 2 of the stage; FP4: K % 64 == 0, so
      // the last stage may be short
      const uint32_t in = (uint32_t)st * 2048 + (u & 1) * 1024 + lane * 16;
      off = in < 16 * rb ? (u >> 1) * 16 * rb + in : kOut;
    } else {
      const uint32_t r = 8 * u + (lane >> 3);
      const uint32_t in = (uint32_t)st * 128 + ((lane & 7) ^ (r & 7)) * 16;
      off = in < rb ? r * rb + in : kOut;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(w.r, (MOE_LDS void *)(lds + u * 1024), 16, off, 0, 0,
                                             2);
  }
}

// A lane's operand from the stage: row block b, half f.  Lane l: r = l % 16
// (weight row), q = l / 16.  It holds the row's 16 bytes 4f + q of 8, i.e. for
// both sides of the product, inputs
//   BF16  32f + 8q .. +7         MX8  64f + 16q .. +15
//   FP4   128f + 32q .. +31, the span of one scale byte
template <int F, bool TILED>
__device__ __forceinline__ u32x4 w_operand(const uint8_t *lds, int b, int f, int lane) {
  const int r = lane & 15, q = lane >> 4;
  if constexpr (!TILED) {
    return *(const u32x4 *)(lds + b * 2048 + r * 128 + (((4 * f + q) ^ (r & 7)) * 16));
  } else if constexpr (F == F_FP4 || F == F_MX4) {
    // four 64-input tiles of 512 bytes; 8-byte pieces 2 (q % 2) and the next of tile 2f + q / 2
    const uint8_t *p = lds + b * 2048 + (2 * f + (q >> 1)) * 512 + ((2 * (q & 1)) * 16 + r) * 8;
    const u32x2 lo = *(const u32x2 *)p, hi = *(const u32x2 *)(p + 128);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  } else {
    return *(const u32x4 *)(lds + b * 2048 + f * 1024 + lane * 16);
  }
}

// FP4 scales.  Eight scale bytes of a row go with a stage of it; loaded stage
// by stage they touch as many cache lines as the weights and cost 20 % of the
// stream, so those of the tile's rows are first copied to LDS, SW bytes a row
// (SW = 256: 31 stages; 64: 7): row layout from the row's first byte rounded
// down to four, its 16-byte pieces permuted so that a half-wave's 16 rows lie in
// distinct banks (unpermuted, a quarter of the LDS cycles were conflicts);
// tiled layout as the row blocks lie, 16 SW bytes each.
template <int F> constexpr bool is_fp4() { return F == F_FP4 || F == F_MX4; }

template <int SW>
__device__ __forceinline__ int scale_swizzle(int r) {
  return SW == 256 ? r & 15 : r >> 2 & 3;
}

// One wave's share (of W = SW / 64 waves) of a source's 32 rows, inputs k0 ...
template <bool TILED, int SW>
__device__ __forceinline__ void copy_scales(const WSrc &w, int K, int k0, int wave, int lane,
                                            uint8_t *lds) {
  constexpr int W = SW / 64;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = wave + W * i;                // 1 KB unit
    uint32_t off;
    if constexpr (TILED) {
      const uint32_t in = (uint32_t)k0 / 2 + (u % W) * 1024 + lane * 16;
      off = in < (uint32_t)K / 2 ? (u / W) * (K / 2) + in : kOut;
    } else {
      const int r = u * (1024 / SW) + lane / (SW / 16);
      const uint32_t row = r * (K / 32);
      const uint32_t at =
          ((row + k0 / 32) & ~3u) + (lane % (SW / 16) ^ scale_swizzle<SW>(r)) * 16;
      off = at < row + K / 32 ? at : kOut;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(w.rs, (MOE_LDS void *)(lds + u * 1024), 16, off, 0, 0,
                                             0);
  }
}
// The scale byte of row block b's row l % 16 for its 32 inputs of half `half`
// (of 128 inputs, from the copied span's start k0); 0 past the row's end.  There
// codes and tokens are zeros, but the copied piece goes on with the next row's
// scales, of which a NaN (0xFF) would not vanish in the product (tiled layout: a
// piece ends with its row block's scales).
template <bool TILED, int SW>
__device__ __forceinline__ uint32_t scale_byte(const uint8_t *lds, int K, int k0, int b, int half,
                                               int lane) {
  const int r = 16 * b + (lane & 15), q = lane >> 4;
  if (TILED) return lds[b * 16 * SW + (2 * half + (q >> 1)) * 32 + (lane & 15) * 2 + (q & 1)];
  const int o = ((r * (K / 32) + k0 / 32) & 3) + half * 4 + q;
  const uint32_t v = lds[r * SW + (o ^ scale_swizzle<SW>(r) << 4)];
  return k0 + 128 * half + 32 * q < K ? v : 0u;
}

// ---------------------------------------------------------------------------
// Token rows: a lane's operand of its row (token l % 16) over a stage.  HILO:
// a second bf16 matrix whose values add to the first's.
template <int F, bool HILO> struct Tokens {
  static constexpr int kV = F == F_F32 ? 1 : F == F_BF16 || F == F_MX8 ? 2 : F == F_MX4 ? 4 : 8;
  static constexpr int kS = F == F_MX4 ? 2 : F == F_MX8 ? 1 : 0;
  static constexpr int kLoads = kV * (HILO ? 2 : 1) + kS;
  u32x4 v[kV * (HILO ? 2 : 1)];
  uint32_t s[kS ? kS : 1];
};
struct TSrc {
  rsrc_t r, r2;                                // r2: low halves (HILO) or scales (MX)
};
// row: the lane's row of the [*, K] matrix; out: kOut for a token not there.
template <int F, bool HILO>
__device__ __forceinline__ void load_tokens(Tokens<F, HILO> &a, const TSrc &src, int K, int lane,
                                            uint32_t row, int st, uint32_t out) {
  const uint32_t q = lane >> 4;
  if constexpr (F == F_F32) {
    const int k0 = st * 16 + 4 * q;
    if (K % 4 == 0) {
      a.v[0] = load16(src.r, (k0 < K ? (row * K + k0) * 4 : kOut) | out);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a.v[0][i] = load4(src.r, (k0 + i < K ? (row * K + k0 + i) * 4 : kOut) | out);
    }
  } else if constexpr (F == F_BF16) {
    const uint32_t off = (row * K + st * 64 + q * 8) * 2;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      a.v[f] = load16(src.r, (off + 64 * f) | out);
      if constexpr (HILO) a.v[2 + f] = load16(src.r2, (off + 64 * f) | out);
    }
  } else if constexpr (F == F_FP4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = (2 * st + h) * 128 + (int)q * 32;
      const uint32_t here = (k0 < K ? 0 : kOut) | out;
      const uint32_t off = (row * K + k0) * 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.v[4 * h + i] = load16(src.r, (off + 16 * i) | here);
        if constexpr (HILO) a.v[8 + 4 * h + i] = load16(src.r2, (off + 16 * i) | here);
      }
    }
  } else {
    constexpr int H = F == F_MX4 ? 2 : 1;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int k0 = (H * st + h) * 128;
      const uint32_t here = (k0 < K ? 0 : kOut) | out;
      const uint32_t off = row * K + k0 + q * 16;
      a.v[2 * h] = load16(src.r, off | here);
      a.v[2 * h + 1] = load16(src.r, (off + 64) | here);
      a.s[h] = load1(src.r2, (row * (K / 32) + k0 / 32 + q) | here);
    }
  }
}

__device__ __forceinline__ f32x4 mma16(const u32x4 &a, const u32x4 &b, const f32x4 &acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ i32x8 wide(const u32x4 &a, const u32x4 &b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3],
               (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// acc += tokens x the 16 rows of row block b over one stage; scl: the source's
// FP4 scales in LDS, `half` the stage's first half in them; s8: the FP8 scale.
template <int F, bool TILED, bool HILO, int SW>
__device__ __forceinline__ void stage_mma(f32x4 &acc, const Tokens<F, HILO> &a, uint32_t s8,
                                          const uint8_t *scl, int K, int k0, int half,
                                          const uint8_t *lds, int b, int lane) {
  if constexpr (F == F_BF16) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const u32x4 w = w_operand<F, TILED>(lds, b, f, lane);
      acc = mma16(a.v[f], w, acc);
      if constexpr (HILO) acc = mma16(a.v[2 + f], w, acc);
    }
  } else if constexpr (F == F_FP4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 codes = w_operand<F, TILED>(lds, b, h, lane);
      const float scale = __uint_as_float(scale_byte<TILED, SW>(scl, K, k0, b, half + h, lane) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 0);
        const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 1);
        const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 2);
        const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 3);
        const u32x4 w = __builtin_bit_cast(
            u32x4, bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]});
        acc = mma16(a.v[4 * h + i], w, acc);
        if constexpr (HILO) acc = mma16(a.v[8 + 4 * h + i], w, acc);
      }
    }
  } else if constexpr (F == F_MX4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          wide(a.v[2 * h], a.v[2 * h + 1]), wide(w_operand<F, TILED>(lds, b, h, lane), u32x4{}),
          acc, 0, 4, 0, (int)a.s[h], 0, (int)scale_byte<TILED, SW>(scl, K, k0, b, half + h, lane));
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        wide(a.v[0], a.v[1]),
        wide(w_operand<F, TILED>(lds, b, 0, lane), w_operand<F, TILED>(lds, b, 1, lane)), acc, 0, 0,
        0, (int)a.s[0], 0, (int)s8);
  }
}

// fp32 layers: a lane's four inputs 16 st + 4q of row block b's row l % 16.
__device__ __forceinline__ u32x4 w_direct(const WSrc &w, int K, int lane, int b, int st) {
  const uint32_t r = 16 * b + (lane & 15), k0 = st * 16 + 4 * (lane >> 4);
  if (K % 4 == 0) return load16(w.r, (int)k0 < K ? (r * K + k0) * 4 : kOut);
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = load4(w.r, (int)k0 + i < K ? (r * K + k0 + i) * 4 : kOut);
  return v;
}

// The wave's tile of products: acc[s][b] = tokens x row block b of source s,
// over stages wave, wave + waves, ..., two stages in flight.  ring0 / ring1: the
// wave's two slots of 4 NB KB; scales: 64 SW bytes (FP4, NB = 2), shared by the
// waves of the tile (four of them for SW = 256, and all call together; one for
// SW = 64).
template <int F, bool TILED, bool HILO, int NB, int SW = 256>
__device__ __forceinline__ void tile_dot(f32x4 (&acc)[2][NB], const TSrc &ts, const WSrc (&ws)[2],
                                         int K, int lane, uint32_t row, bool there, int wave,
                                         int waves, uint8_t *ring0, uint8_t *ring1,
                                         uint8_t *scales) {
  const uint32_t out = there ? 0u : kOut;
  constexpr int KST = stage_inputs<F>();
  const int nst = (K + KST - 1) / KST;
  if constexpr (F == F_F32) {
    (void)ring0; (void)ring1; (void)scales;
    for (int st = wave; st < nst; st += waves) {
      Tokens<F, HILO> a;
      load_tokens<F, HILO>(a, ts, K, lane, row, st, out);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const u32x4 w = w_direct(ws[s], K, lane, b, st);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[s][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __uint_as_float(a.v[0][i]), __uint_as_float(w[i]), acc[s][b], 0, 0, 0);
        }
    }
  } else {
    constexpr int VM = 4 * NB + Tokens<F, HILO>::kLoads + (F == F_MX8 ? 2 : 0);
    static_assert(2 * VM <= 63, "vmcnt holds 6 bits");
    static_assert(!is_fp4<F>() || NB == 2, "32 rows of scales a source");
    constexpr int SPAN = is_fp4<F>() ? SW / 8 - 1 : 1 << 30;   // stages
    Tokens<F, HILO> a[2];
    uint32_t s8[2][2];
    // stages lo .. hi - 1 (whose scales are in LDS)
    for (int lo = 0; lo < nst; lo += SPAN) {
      const int hi = nst - lo > SPAN ? lo + SPAN : nst;
      if constexpr (is_fp4<F>()) {
        // every wave is done with the last scales
        if (lo > 0 && SW == 256) __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s)
          copy_scales<TILED, SW>(ws[s], K, lo * KST, wave, lane, scales + s * 32 * SW);
      }
      auto issue = [&](int p, int st) {
        uint8_t *lds = p ? ring1 : ring0;
        load_tokens<F, HILO>(a[p], ts, K, lane, row, st, out);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if constexpr (F == F_MX8) s8[p][s] = load1(ws[s].rs, st);
          copy_stage<F, TILED, NB>(ws[s], K, lane, st, lds + s * NB * 2048);
        }
        // keep the loads here: the scheduler otherwise moves them behind the
        // next products
        __builtin_amdgcn_sched_barrier(0);
      };
      auto compute = [&](int p, int st) {
        const uint8_t *lds = p ? ring1 : ring0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            stage_mma<F, TILED, HILO, SW>(acc[s][b], a[p], F == F_MX8 ? s8[p][s] : 0,
                                      scales + s * 32 * SW, K, lo * KST, 2 * (st - lo),
                                      lds + s * NB * 2048, b, lane);
        // the slot's reads are done before a copy may land in it again
        __builtin_amdgcn_s_waitcnt(0xC07F);    // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
      };
      // at most n younger loads outstanding; no LDS read moves above
#define MOE_LANDED(n)                                \
      __builtin_amdgcn_s_waitcnt(MOE_VMCNT(n));      \
      asm volatile("" ::: "memory");                 \
      __builtin_amdgcn_sched_barrier(0)
      int st = lo + wave;
      const int n = hi > st ? (hi - st + waves - 1) / waves : 0;
      if (n > 0) issue(0, st);
      if (n > 1) issue(1, st + waves);
      if constexpr (is_fp4<F>()) {
        // the scales are older than the stages issued
        if (n > 1) { MOE_LANDED(2 * VM); } else { MOE_LANDED(0); }
        if (SW == 256) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      if (n > 1) {
        int i = 0;
        for (; i + 3 < n; i += 2, st += 2 * waves) {
          MOE_LANDED(VM);
          compute(0, st);
          issue(0, st + 2 * waves);
          MOE_LANDED(VM);
          compute(1, st + waves);
          issue(1, st + 3 * waves);
        }
        MOE_LANDED(VM);
        compute(0, st);
        if (i + 2 < n) issue(0, st + 2 * waves);
        MOE_LANDED(0);
        compute(1, st + waves);
        if (i + 2 < n) compute(0, st + 2 * waves);
      } else if (n == 1) {
        MOE_LANDED(0);
        compute(0, st);
      }
#undef MOE_LANDED
    }
  }
}

// The waves' 16 x 16 products go through LDS: element 16 row + column of block
// (s, b), each wave in its own region of 2 NB KB.
template <int NB>
__device__ __forceinline__ void put_partial(float *mine, const f32x4 (&acc)[2][NB], int lane) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mine[(s * NB + b) * 256 + ((lane >> 4) * 4 + i) * 16 + (lane & 15)] = acc[s][b][i];
}

// H as two bf16 whose sum holds 16 bits of the fp32 value, so that the down
// product sees more than a bf16's 8 (the second MFMA is free here).  A value
// that overflows bf16 keeps its infinity.
__device__ __forceinline__ void store_hilo(bf16 *hi, bf16 *lo, int64_t at, float v) {
  const bf16 h = (bf16)v;
  const float hf = (float)h;
  hi[at] = h;
  lo[at] = (__float_as_uint(hf) & 0x7F800000u) == 0x7F800000u ? (bf16)0.f : (bf16)(v - hf);
}

// SwiGLU of a gate / up pair, clamped by comparisons that a NaN passes (a
// minimum or maximum would put the bound in its place).  H of an fp32 layer is
// stored as it comes, so its exponential and division are the accurate ones; the
// others round H to 16 bits or fewer and take the hardware's (swiglu_pair).
template <int F>
__device__ __forceinline__ float swiglu_few(float g, float u, float L) {
  if (L > 0.f) {
    g = g > L ? L : g;
    u = u > L ? L : (u < -L ? -L : u);
  }
  if constexpr (F == F_F32) return g / (1.f + expf(-g)) * u;
  else return swiglu_pair(g, u, 0.f);
}

// MXFP8 (OCP MX): what a value adds to its block's maximum magnitude, the
// block's shared exponent, and the element to encode.  E4M3 has no infinity, and
// a maximum over NaN or infinities gives no exponent: those values take the NaN
// code each and leave the block's exponent to the others.
__device__ __forceinline__ float mx_magnitude(float v) {
  const float m = fabsf(v);
  return m < INFINITY ? m : 0.f;
}
__device__ __forceinline__ int mx_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int ex;
  frexpf(amax, &ex);
  const int X = ex - 1 - 8;
  return X < -127 ? -127 : (X > 127 ? 127 : X);
}
__device__ __forceinline__ float mx_element(float v, int X) {
  return fabsf(v) < INFINITY ? fminf(fmaxf(ldexpf(v, -X), -448.f), 448.f) : NAN;
}

// ---------------------------------------------------------------------------
// few_scores: partial gate logits and, for MXFP8 layers, the codes of x.  A
// workgroup takes 16 experts and one of KS parts of the inputs, its four waves
// splitting those, each with one burst of loads: latency, not bandwidth, is
// what the gate matrix (a few MB) costs.
// Logits of 16 experts from n0 for every token over stages first .. end - 1, of
// which wave kw of four takes every fourth: red[token * 16 + expert].
template <int F>
__device__ __forceinline__ void score_block(const FewArgs &a, int n0, int first, int end, int kw,
                                            int lane, float *red) {
  constexpr int DEPTH = 4;
  constexpr int es = F == F_F32 ? 4 : 2;
  const int d = a.d, T = a.T, r = lane & 15, q = lane >> 4;
  const TSrc ts = {resource(a.x, (int64_t)T * d * es), resource(a.x, 0)};
  const int have = a.E - n0 < 16 ? a.E - n0 : 16;
  const WSrc w = {resource((const uint8_t *)a.gate_w + (int64_t)n0 * d * es, (int64_t)have * d * es),
                  resource(a.gate_w, 0)};
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  Tokens<F, false> tk[DEPTH];
  u32x4 wv[DEPTH][2];
  auto load = [&](int p, int st) {
    load_tokens<F, false>(tk[p], ts, d, lane, r, st, st < end && r < T ? 0u : kOut);
    if constexpr (F == F_F32) {
      wv[p][0] = w_direct(w, d, lane, 0, st);
    } else {
      const uint32_t off = ((uint32_t)r * d + st * 64 + q * 8) * 2;
      wv[p][0] = load16(w.r, st < end ? off : kOut);
      wv[p][1] = load16(w.r, st < end ? off + 64 : kOut);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // whole bursts of DEPTH stages a wave; tokens past the end read as zeros
  for (int st = first + kw; st < end; st += 4 * DEPTH) {
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) load(p, st + 4 * p);
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) {
      if constexpr (F == F_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(
              __uint_as_float(tk[p].v[0][i]),
              st + 4 * p < end ? __uint_as_float(wv[p][0][i]) : 0.f, acc, 0, 0, 0);
      } else {
        acc = mma16(tk[p].v[0], wv[p][0], acc);
        acc = mma16(tk[p].v[1], wv[p][1], acc);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[(q * 4 + i) * 16 + r] = acc[i];
}

template <int F>
__global__ __launch_bounds__(256) void few_scores(const FewArgs a) {
  __shared__ float red[4 * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d = a.d, T = a.T;
  int item = blockIdx.x;
  if (item < a.score_items) {
    constexpr int KST = stage_inputs<F>();
    const int part = item % a.KS, n0 = item / a.KS * 16, nst = (d + KST - 1) / KST;
    score_block<F>(a, n0, (int)((int64_t)nst * part / a.KS),
                   (int)((int64_t)nst * (part + 1) / a.KS), wave, lane, red + wave * 256);
    __syncthreads();
    const int t = threadIdx.x >> 4, e = n0 + (threadIdx.x & 15);
    if (t < T && e < a.E)
      a.scores[((int64_t)part * T + t) * a.E + e] =
          ((red[threadIdx.x] + red[256 + threadIdx.x]) + red[512 + threadIdx.x]) +
          red[768 + threadIdx.x];
    return;
  }
  item -= a.score_items;
  if constexpr (F == F_BF16) {
    const int i = item * (int)blockDim.x + (int)threadIdx.x;
    if (!a.xq || i >= T * d / 32) return;
    const u32x4 *p = (const u32x4 *)((const bf16 *)a.x + (int64_t)i * 32);
    float v[32], amax = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bf16x8 w = __builtin_bit_cast(bf16x8, p[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[8 * c + j] = (float)w[j];
        amax = fmaxf(amax, mx_magnitude(v[8 * c + j]));
      }
    }
    const int X = mx_exponent(amax);
    a.xq_scales[i] = (uint8_t)(X + 127);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      int word = __builtin_amdgcn_cvt_pk_fp8_f32(mx_element(v[4 * j], X),
                                                 mx_element(v[4 * j + 1], X), 0, false);
      w[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(mx_element(v[4 * j + 2], X),
                                                       mx_element(v[4 * j + 3], X), word, true);
    }
    u32x4 *o = (u32x4 *)(a.xq + (int64_t)i * 32);
    o[0] = u32x4{w[0], w[1], w[2], w[3]};
    o[1] = u32x4{w[4], w[5], w[6], w[7]};
  }
}

// ---------------------------------------------------------------------------
// Selection of one token by one wave, as route.hip's select_token: the same
// affinities, bias, group limit, top-k and ties, with groups of any size (a
// group of one expert scores by it alone).  Lane l holds experts
// l*EPL .. l*EPL+EPL-1.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max_step(float v) {
  const int ninf = __float_as_int(-INFINITY);
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(ninf, __float_as_int(v), CTRL, ROWS,
                                                             0xF, false)));
}
// Maximum over the wave, in every lane: row shifts 1, 2, 4, 8, then the row
// broadcasts, then lane 63's value.
__device__ __forceinline__ float wave_max_dpp(float v) {
  v = dpp_max_step<0x111, 0xF>(v);
  v = dpp_max_step<0x112, 0xF>(v);
  v = dpp_max_step<0x114, 0xF>(v);
  v = dpp_max_step<0x118, 0xF>(v);
  v = dpp_max_step<0x142, 0xA>(v);
  v = dpp_max_step<0x143, 0xC>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// A wave's LDS accesses stay in order across this.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Group limit where a group is no power of two of whole lanes, in LDS: `row` holds the
// token's E keys and becomes 1 for each of the G groups that stays, 0 for the
// others; `score` takes the groups' scores.  A lane takes groups lane, lane + 64,
// ...; the loops stay loops, or the selection's registers would spill.
__device__ __forceinline__ void limit_groups(const FewArgs &a, int lane, float *row, float *score) {
  const int G = a.G, size = a.E / G;
  wave_order();
#pragma unroll 1
  for (int g = lane; g < G; g += 64) {
    float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll 1
    for (int e = g * size; e < (g + 1) * size; ++e) {
      const float v = row[e];
      if (v > a1) { a2 = a1; a1 = v; } else if (v > a2) { a2 = v; }
    }
    score[g] = a.bias && size > 1 ? a1 + a2 : a1;
  }
  wave_order();
#pragma unroll 1
  for (int g = lane; g < G; g += 64) {
    const float own = score[g];
    int rank = 0;
#pragma unroll 1
    for (int gg = 0; gg < G; ++gg) {
      const float v = score[gg];
      rank += (v > own) || (v == own && gg < g);
    }
    row[g] = rank < a.kept ? 1.f : 0.f;
  }
  wave_order();
}

template <int EPL, bool ODD>
__device__ __forceinline__ void select_few(const FewArgs &a, int t, int lane, float *out_w,
                                           int32_t *out_e, float *scores,
                                           const float *gate_bias) {
  const int E = a.E;
  float s[EPL], key[EPL], bias[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane * EPL + j;
    s[j] = e < E ? scores[t * E + e] : 0.f;
    bias[j] = a.bias && e < E ? gate_bias[e] : 0.f;
  }
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, lane * EPL + j < E ? s[j] : -INFINITY);
    m = wave_max_dpp(m);
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      s[j] = lane * EPL + j < E ? expf(s[j] - m) : 0.f;
      part += s[j];
    }
    const float inv = 1.f / wave_sum(part);
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] *= inv;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    key[j] = a.bias ? s[j] + bias[j] : s[j];
    // NaN scores come last
    if (lane * EPL + j >= E || key[j] != key[j]) key[j] = -INFINITY;
  }
  if constexpr (ODD) {
    float *row = scores + t * E;               // read by this wave alone, and no more
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane * EPL + j < E) row[lane * EPL + j] = key[j];
    limit_groups(a, lane, row, scores + (kRows + t) * 512);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane * EPL + j;
      if (e < E && row[e / (E / a.G)] == 0.f) key[j] = -INFINITY;
    }
  } else if (a.G > 1) {
    const int size = E / a.G, lpg = size / EPL;  // experts and lanes of a group
    float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float v = key[j];
      if (v > a1) { a2 = a1; a1 = v; } else if (v > a2) { a2 = v; }
    }
#define MOE_GROUP_MERGE(M)                                              \
    if (lpg > M) {                                                      \
      const float b1 = xor_lane<M>(a1), b2 = xor_lane<M>(a2);           \
      const float hi = fmaxf(a1, b1), lo = fminf(a1, b1);               \
      a2 = fmaxf(lo, fmaxf(a2, b2));                                    \
      a1 = hi;                                                          \
    }
    MOE_GROUP_MERGE(1) MOE_GROUP_MERGE(2) MOE_GROUP_MERGE(4)
    MOE_GROUP_MERGE(8) MOE_GROUP_MERGE(16) MOE_GROUP_MERGE(32)
#undef MOE_GROUP_MERGE
    const float gs = a.bias && size > 1 ? a1 + a2 : a1;
    const int g = lane / lpg;
    int rank = 0;
    for (int gg = 0; gg < a.G; ++gg) {
      const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gs), gg * lpg));
      rank += (v > gs) || (v == gs && gg < g);
    }
    if (g >= a.G || rank >= a.kept) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = -INFINITY;
    }
  }
  unsigned taken = 0;
  int my_e = 0;
  float my_s = 0.f, ssum = 0.f;
  for (int r = 0; r < a.k; ++r) {
    float bv = -INFINITY, bs = 0.f;
    int bj = -1;                               // the lane's best untaken slot, lowest first
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane * EPL + j < E && !((taken >> j) & 1u) && (bj < 0 || key[j] > bv)) {
        bv = key[j];
        bs = s[j];
        bj = j;
      }
    const float m = wave_max_dpp(bv);
    // k <= E: some lane has an untaken expert at the maximum; lowest lane = lowest id
    const int owner = __builtin_ctzll(__ballot(bj >= 0 && bv == m));
    const int slot = __builtin_amdgcn_readlane(bj, owner);
    const float sv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bs), owner));
    if (lane == owner) taken |= 1u << slot;
    if (lane == r) { my_e = owner * EPL + slot; my_s = sv; }
    ssum += sv;
  }
  if (lane < a.k) {
    float w = my_s;
    if (a.renorm) w = w / ssum;
    out_e[t * a.k + lane] = my_e;
    out_w[t * a.k + lane] = w * a.route_scale;
  }
}

template <bool ODD>
__device__ __forceinline__ void select_any(const FewArgs &a, int t, int lane, float *w, int32_t *e,
                                           float *scores, const float *bias) {
  switch ((a.E + 63) / 64) {
    case 1: return select_few<1, ODD>(a, t, lane, w, e, scores, bias);
    case 2: return select_few<2, ODD>(a, t, lane, w, e, scores, bias);
    case 3: return select_few<3, ODD>(a, t, lane, w, e, scores, bias);
    case 4: return select_few<4, ODD>(a, t, lane, w, e, scores, bias);
    case 5: return select_few<5, ODD>(a, t, lane, w, e, scores, bias);
    case 6: return select_few<6, ODD>(a, t, lane, w, e, scores, bias);
    case 7: return select_few<7, ODD>(a, t, lane, w, e, scores, bias);
    default: return select_few<8, ODD>(a, t, lane, w, e, scores, bias);
  }
}

// Routes all tokens and writes the plan: the distinct chosen experts ("slots",
// by first appearance in (token, choice) order), for each slot and token the H
// row (the pair's number t*k + j; -1: not chosen) and the gate value (summed
// where a token has the expert twice), and for each token the choices that
// hold a row.  One workgroup of 16 waves; a thread per pair.
struct PlanScratch {
  float w[256];
  int32_t e[256];
  int32_t lead[1024];                          // per expert: its first pair, then its slot
  int32_t misc[8];
  uint32_t mask[kRows];
  float cell_w[256 * kRows];
  int16_t cell_row[256 * kRows];
};
template <int F, bool ODD>
__device__ __forceinline__ void make_plan(const FewArgs &a, PlanScratch &p, float *scores) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int T = a.T, k = a.k, E = a.E, pairs = T * k;
  if (tid == 0) p.misc[0] = 0;
  if (tid < kRows) p.mask[tid] = 0;
  for (int i = tid; i < pairs * kRows; i += 1024) {
    p.cell_w[i] = 0.f;
    p.cell_row[i] = -1;
  }
  if (a.route_mode == MOE_ROUTE_LEARNED) {
    // affinities of all tokens by all threads (softmax: the logits), the parts
    // of a logit added in order; then a wave per token
    const int n = T * E;
    float *bias = (float *)p.lead;             // until the leaders
    if (a.bias)
      for (int i = tid; i < E; i += 1024) bias[i] = a.bias[i];
    float *red = scores + kRows * 512;
    if (a.small_gate) {                        // four waves a block of 16 experts
      if (wave / 4 * 16 < E)
        score_block<F>(a, wave / 4 * 16, 0, (a.d + stage_inputs<F>() - 1) / stage_inputs<F>(),
                       wave & 3, lane, red + wave * 256);
      __syncthreads();
    }
    for (int i = tid; i < n; i += 1024) {
      float z;
      if (a.small_gate) {
        const int t = i / E, e = i - t * E;
        const float *r = red + e / 16 * 1024 + t * 16 + e % 16;
        z = ((r[0] + r[256]) + r[512]) + r[768];
      } else {
        float part[kLogitParts];
#pragma unroll
        for (int q = 0; q < kLogitParts; ++q)
          part[q] = q < a.KS ? a.scores[(int64_t)q * n + i] : 0.f;
        z = part[0];
#pragma unroll
        for (int q = 1; q < kLogitParts; ++q) z += part[q];
      }
      if (a.score == MOE_SCORE_SIGMOID) z = 1.f / (1.f + expf(-z));
      else if (a.score == MOE_SCORE_SQRTSOFTPLUS)
        z = sqrtf(fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
      scores[i] = z;
    }
    __syncthreads();
    for (int t = wave; t < T; t += 16) select_any<ODD>(a, t, lane, p.w, p.e, scores, bias);
    __syncthreads();
  } else {
    __syncthreads();
    if (tid < pairs) {
      const int t = tid / k, j = tid - t * k;
      bool ok;
      int e;
      if (a.route_mode == MOE_ROUTE_HASH) {
        const int64_t id = a.token_ids[t];
        ok = id >= 0 && id < a.vocab;
        e = a.tid2eid[(ok ? id : 0) * k + j];
      } else {
        const int64_t prev = a.token_ids[2 * t], cur = a.token_ids[2 * t + 1];
        ok = prev >= -1 && prev < a.vocab && cur >= 0 && cur < a.vocab;
        const int64_t u = ok && prev >= 0 ? prev : a.vocab, v = ok ? cur : 0;
        e = (int)((u * a.primes[j] + v) % E);
      }
      p.e[tid] = e;
      p.w[tid] = ok ? a.route_scale / (float)k : 0.f;
      const int bad = (ok ? 0 : (int)MOE_FLAG_TOKEN_ID_RANGE) |
                      (e >= 0 && e < E ? 0 : (int)MOE_FLAG_EXPERT_RANGE);
      if (bad) atomicOr(&p.misc[0], bad);
    }
    __syncthreads();
  }
  const int e = tid < pairs ? p.e[tid] : -1;
  const bool in = e >= 0 && e < E;             // a table may hold ids past E: dropped
  if (in) p.lead[e] = INT_MAX;
  __syncthreads();
  if (in) atomicMin(&p.lead[e], tid);
  __syncthreads();
  const bool first = in && p.lead[e] == tid;
  // slot = number of earlier leaders; the pairs (<= 256) are in the first four waves
  const uint64_t vote = __ballot(first);
  if (lane == 0 && wave < 4) p.misc[1 + wave] = __popcll(vote);
  __syncthreads();
  int slot = __popcll(vote & ((1ull << lane) - 1)), slots = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) slot += p.misc[1 + w];
    slots += p.misc[1 + w];
  }
  if (first) {
    p.lead[e] = slot;
    a.plan_expert[slot] = e;
  }
  if (tid < pairs) {
    a.out_w[tid] = p.w[tid];
    a.out_e[tid] = e;
  }
  if (tid == 0) {
    a.plan_slots[0] = slots;
    a.flags[0] = (uint32_t)p.misc[0];
  }
  __syncthreads();
  if (in) {
    const int t = tid / k, j = tid - t * k;
    float w = 0.f;
    bool mine = true;                          // the token's first choice of this expert
    for (int i = 0; i < k; ++i)
      if (p.e[t * k + i] == e) {
        mine = mine && i >= j;
        w += p.w[t * k + i];
      }
    if (mine) {
      const int cell = p.lead[e] * kRows + t;
      p.cell_w[cell] = w;
      p.cell_row[cell] = (int16_t)tid;
      atomicOr(&p.mask[t], 1u << j);
    }
  }
  __syncthreads();
  for (int i = tid; i < slots * kRows; i += 1024) {
    a.plan_w[i] = p.cell_w[i];
    a.plan_row[i] = p.cell_row[i];
  }
  if (tid < T) a.plan_mask[tid] = (int32_t)p.mask[tid];
}

// ---------------------------------------------------------------------------
// Tile of gate|up: 16 NB columns of H; the wave's partial products to `mine`.
template <int F, bool TILED, int NB>
__device__ __forceinline__ void up_tile(const FewArgs &a, const TSrc &xs, const void *wg,
                                        const void *wu, const uint8_t *sg, const uint8_t *su,
                                        int n0, uint32_t row, bool there, int wave, int waves,
                                        int lane, uint8_t *ring0, uint8_t *ring1, uint8_t *scales,
                                        float *mine) {
  const WSrc ws[2] = {w_source<F>(wg, sg, a.I, a.d, n0, 16 * NB),
                      w_source<F>(wu, su, a.I, a.d, n0, 16 * NB)};
  f32x4 acc[2][NB];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[s][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  tile_dot<F, TILED, false, NB>(acc, xs, ws, a.d, lane, row, there, wave, waves, ring0, ring1,
                                scales);
  put_partial<NB>(mine, acc, lane);
}

// few_plan: workgroup 0 routes; the others stream the shared expert's gate|up,
// 16 columns each, 16 waves splitting the inputs.  ODD: groups through LDS, a
// kernel of its own, since that code beside the lanes' one slowed every layer (18.8
// -> 20.2 us for a 3-token layer of 16 experts without groups).
template <int F, bool TILED, bool ODD>
__global__ __launch_bounds__(1024) void few_plan(const FewArgs a) {
  constexpr int SLOT = F == F_F32 ? 2048 : 4096;
  constexpr int PLAN = (int)sizeof(PlanScratch);
  __shared__ __attribute__((aligned(1024))) uint8_t R0[16 * SLOT > PLAN ? 16 * SLOT : PLAN];
  __shared__ __attribute__((aligned(1024))) uint8_t R1[16 * 4096];
  static_assert(sizeof(R1) >= kRows * 512 * 4 + 16 * 256 * 4, "affinities, logits of a small gate");
  static_assert(sizeof(R1) >= 2 * kRows * 512 * 4, "affinities, scores of odd groups");
  if (blockIdx.x == 0) {
    make_plan<F, ODD>(a, *(PlanScratch *)R0, (float *)R1);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int es = F == F_F32 ? 4 : 2;
  const int n0 = (blockIdx.x - 1) * 16, t0 = lane & 15;
  const TSrc xs = {resource(a.x, (int64_t)a.T * a.d * es), resource(a.x, 0)};
  float *red = (float *)R0;
  up_tile<F, TILED, 1>(a, xs, a.sh_gate, a.sh_up, nullptr, nullptr, n0, t0, t0 < a.T, wave, 16, lane,
                       R0 + wave * SLOT, F == F_F32 ? R0 : R1 + wave * SLOT, nullptr,
                       red + wave * (SLOT / 4));
  __syncthreads();
  for (int e = threadIdx.x; e < 256; e += 1024) {
    const int t = e >> 4, n = n0 + (e & 15);
    if (t >= a.T || n >= a.I) continue;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      g += red[w * (SLOT / 4) + e];
      u += red[w * (SLOT / 4) + 256 + e];
    }
    const float v = swiglu_few<F>(g, u, a.limit);
    const int64_t at = (int64_t)(a.T * a.k + t) * a.I + n;
    if constexpr (F == F_F32) ((float *)a.h)[at] = v;
    else store_hilo((bf16 *)a.h, (bf16 *)a.h_lo, at, v);
  }
}

// LDS of the up and down launches: two ring slots of 8 KB a wave and the FP4
// scales, 80 KB, so that two workgroups share a CU and cover each other's
// starts and ends.
#define MOE_FEW_LDS(F)                                                                        \
  constexpr int SLOT = F == F_F32 ? 4096 : 8192;                                              \
  __shared__ __attribute__((aligned(1024))) uint8_t R0[4 * SLOT];                             \
  __shared__ __attribute__((aligned(1024))) uint8_t R1[F == F_F32 ? 16 : 4 * SLOT];           \
  __shared__ __attribute__((aligned(1024))) uint8_t SC[is_fp4<F>() ? 16384 : 16];             \
  float *red = (float *)R0;                                                                   \
  const int lane = threadIdx.x & 63;                                                          \
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);                          \
  uint8_t *ring0 = R0 + wave * SLOT, *ring1 = F == F_F32 ? R0 : R1 + wave * SLOT

// few_up: a workgroup takes 32 columns of H of one slot (an MXFP8 scale block),
// its four waves splitting the inputs.
template <int F, bool TILED>
__global__ __launch_bounds__(256, 2) void few_up(const FewArgs a) {
  constexpr bool MX = F == F_MX4 || F == F_MX8;
  constexpr int NB = 2;
  constexpr int es = F == F_F32 ? 4 : 2;
  MOE_FEW_LDS(F);
  const int T = a.T, d = a.d, I = a.I;
  const int blocks = (I + 31) / 32, pairs = T * a.k;
  // a tile's slot, asked for with the number of slots (past it: not used)
  auto slot_of = [&](int tile) {
    const int s = tile / blocks;
    return s < pairs ? s : pairs - 1;
  };
  int expert = a.plan_expert[slot_of(blockIdx.x)];
  int16_t row = a.plan_row[slot_of(blockIdx.x) * kRows + (lane & 15)];
  const int tiles = a.plan_slots[0] * blocks;
  TSrc xs;
  if constexpr (MX) {
    xs.r = resource(a.xq, (int64_t)T * d);
    xs.r2 = resource(a.xq_scales, (int64_t)T * (d / 32));
  } else {
    xs.r = resource(a.x, (int64_t)T * d * es);
    xs.r2 = xs.r;
  }
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int slot = tile / blocks, n0 = (tile - slot * blocks) * 32;
    const int16_t *rows = a.plan_row + slot * kRows;
    const int64_t e = expert;
    const int64_t at = e * ((int64_t)I * row_bytes<F>(d));
    const int64_t sat = e * ((int64_t)I * d / (F == F_MX8 ? 16384 : 32));
    up_tile<F, TILED, NB>(a, xs, (const uint8_t *)a.w_gate + at, (const uint8_t *)a.w_up + at,
                          a.s_gate + sat, a.s_up + sat, n0, lane & 15, row >= 0, wave, 4, lane,
                          ring0, ring1, SC, red + wave * (SLOT / 4));
    expert = a.plan_expert[slot_of(tile + gridDim.x)];
    row = a.plan_row[slot_of(tile + gridDim.x) * kRows + (lane & 15)];
    __syncthreads();
    // a half-wave takes a token's 32 columns
    for (int t = threadIdx.x >> 5; t < kRows; t += 8) {
      const int pair = rows[t], c = lane & 31, n = n0 + c;
      const int el = (c >> 4) * 256 + t * 16 + (c & 15);
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        g += red[w * (SLOT / 4) + el];
        u += red[w * (SLOT / 4) + NB * 256 + el];
      }
      const float v = swiglu_few<F>(g, u, a.limit);
      if constexpr (MX) {
        float amax = mx_magnitude(v);
        amax = fmaxf(amax, xor_lane<1>(amax));
        amax = fmaxf(amax, xor_lane<2>(amax));
        amax = fmaxf(amax, xor_lane<4>(amax));
        amax = fmaxf(amax, xor_lane<8>(amax));
        amax = fmaxf(amax, xor_lane<16>(amax));
        const int X = mx_exponent(amax);
        const int word = __builtin_amdgcn_cvt_pk_fp8_f32(mx_element(v, X), 0.f, 0, false);
        if (pair >= 0) {
          a.hq[(int64_t)pair * I + n] = (uint8_t)word;
          if (c == 0) a.hq_scales[(int64_t)pair * (I / 32) + n0 / 32] = (uint8_t)(X + 127);
        }
      } else if (pair >= 0 && n < I) {
        const int64_t o = (int64_t)pair * I + n;
        if constexpr (F == F_F32) ((float *)a.h)[o] = v;
        else store_hilo((bf16 *)a.h, (bf16 *)a.h_lo, o, v);
      }
    }
    __syncthreads();
  }
}

// Tile of W_down: 64 output columns of one slot; the wave's partial to `mine`.
template <int F, bool TILED, bool HILO, int SW>
__device__ __forceinline__ void down_tile(const FewArgs &a, const TSrc &hs, const void *w,
                                          const uint8_t *sc, int n0, int row, int wave, int waves,
                                          int lane, uint8_t *ring0, uint8_t *ring1, uint8_t *scales,
                                          float *mine) {
  constexpr int NB = 2;
  const WSrc ws[2] = {w_source<F>(w, sc, a.d, a.I, n0, 32), w_source<F>(w, sc, a.d, a.I, n0 + 32, 32)};
  f32x4 acc[2][NB];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[s][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  tile_dot<F, TILED, HILO, NB, SW>(acc, hs, ws, a.I, lane, row < 0 ? 0 : row, row >= 0, wave, waves,
                                   ring0, ring1, scales);
  put_partial<NB>(mine, acc, lane);
}

// few_down: yrows[pair] = w (H[pair] W_down^T) in fp32, rows T*k .. the shared
// expert's.  A tile is 64 columns of one slot, taken by G waves: four, or one
// where the tile is a few stages long (FP4 with I <= 1792: MXFP8 at 16 tokens
// 108 -> 89 us; four waves had one or two stages each).  The shared tiles
// (longer, in bf16, four waves) come first.
// PACK (T <= 8): the two halves of H ride in one operand, MFMA row t the high
// half of token t and row 8 + t the low one, whose products are added at the
// end; more tokens take a second operand.
template <int F, bool TILED, bool PACK, int G>
__global__ __launch_bounds__(256, 2) void few_down(const FewArgs a) {
  constexpr bool MX = F == F_MX4 || F == F_MX8;
  constexpr bool F32 = F == F_F32;
  constexpr int kLow = 8 * 16;                 // the low half's products in a 16 x 16 block
  constexpr int SW = G == 4 ? 256 : 64, PER = 4 / G;
  MOE_FEW_LDS(F);
  const int T = a.T, d = a.d, I = a.I, pairs = T * a.k;
  const int blocks = (d + 63) / 64;
  const int shared = a.has_shared ? blocks : 0;
  // as in few_up
  auto slot_of = [&](int unit) {
    const int s = ((unit - shared) * PER + (G == 1 ? wave : 0)) / blocks;
    return s < 0 ? 0 : s < pairs ? s : pairs - 1;
  };
  int expert = a.plan_expert[slot_of(blockIdx.x)];
  const int tiles = a.plan_slots[0] * blocks;
  const int units = shared + (tiles + PER - 1) / PER;
  const int hrows = pairs + (a.has_shared ? T : 0);
  const int64_t hbytes = (int64_t)hrows * I * (F32 ? 4 : 2);
  // the low halves follow the high ones
  const TSrc hs = {resource(a.h, F32 ? hbytes : 2 * hbytes), resource(F32 ? a.h : a.h_lo, hbytes)};
  const TSrc qs = {resource(a.hq, MX ? (int64_t)pairs * I : 0),
                   resource(a.hq_scales, MX ? (int64_t)pairs * (I / 32) : 0)};
  float *mine = red + wave * (SLOT / 4);
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const bool sh = unit < shared;
    const int tile = sh ? unit : (unit - shared) * PER + (G == 1 ? wave : 0);
    const bool live = sh || tile < tiles;
    const int slot = sh || !live ? 0 : tile / blocks;
    const int n0 = (live ? tile - slot * blocks : 0) * 64;
    const int16_t *rows = a.plan_row + slot * kRows;
    const bool packed = PACK && (sh || !MX);
    const int t = packed ? lane & 7 : lane & 15;
    const int low = packed && (lane & 8) ? hrows : 0;
    if (sh) {
      down_tile<F32 ? F_F32 : F_BF16, TILED && !F32, !F32 && !PACK, 256>(
          a, hs, a.sh_down, nullptr, n0, t < T ? pairs + t + low : -1, wave, 4, lane, ring0, ring1,
          nullptr, mine);
    } else if (live) {
      const int64_t e = __builtin_amdgcn_readfirstlane(expert);
      const int64_t at = e * ((int64_t)d * row_bytes<F>(I));
      const int64_t sat = e * ((int64_t)d * I / (F == F_MX8 ? 16384 : 32));
      const int row = rows[t];
      down_tile<F, TILED, !F32 && !MX && !PACK, SW>(
          a, MX ? qs : hs, (const uint8_t *)a.w_down + at, a.s_down + sat, n0,
          row < 0 ? row : row + low, G == 1 ? 0 : wave, G, lane, ring0, ring1,
          SC + (G == 1 ? wave * 64 * SW : 0), mine);
    }
    expert = a.plan_expert[slot_of(unit + gridDim.x)];
    __syncthreads();
    const bool own = G == 1 && !sh;            // the wave's tile is its own
    if (live)
      for (int tt = own ? 0 : wave; tt < T; tt += own ? 1 : 4) {
        const int pair = sh ? pairs + tt : rows[tt], n = n0 + lane;
        if (pair < 0 || n >= d) continue;
        const int el = (lane >> 4) * 256 + tt * 16 + (lane & 15);
        float v = 0.f;
        for (int w = own ? wave : 0; w < (own ? wave + 1 : 4); ++w) {
          v += red[w * (SLOT / 4) + el];
          if (packed) v += red[w * (SLOT / 4) + el + kLow];
        }
        a.yrows[(int64_t)pair * d + n] = sh ? v : a.plan_w[slot * kRows + tt] * v;
      }
    __syncthreads();
  }
}

// few_combine: y[t] = the sum of the token's rows, in choice order, and the
// shared one.
template <typename T>
__global__ __launch_bounds__(256) void few_combine(const FewArgs a) {
  const int t = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= a.d) return;
  const int left = a.d - n;
  const uint32_t mask = (uint32_t)a.plan_mask[t];
  const bool whole = left >= 4 && a.d % 4 == 0;
  auto row = [&](int r) {
    const float *p = a.yrows + (int64_t)r * a.d + n;
    if (whole) return *(const f32x4 *)p;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < 4 && i < left; ++i) v[i] = p[i];
    return v;
  };
  // eight rows asked for at a time, beside the mask that says which were written,
  // and added in the order of the choices
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 sum = zero, last = zero;
  if (a.has_shared) last = row(a.T * a.k + t);
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    f32x4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j0 + j < a.k ? row(t * a.k + j0 + j) : zero;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += mask >> (j0 + j) & 1u ? v[j] : zero;
  }
  sum += last;
  T *y = (T *)a.y + (int64_t)t * a.d + n;
  for (int i = 0; i < 4 && i < left; ++i) y[i] = (T)sum[i];
}

constexpr int kGroups = 512;                   // resident workgroups of four waves: two a CU

template <int F, bool TILED>
hipError_t run_few(FewArgs a, hipStream_t s) {
  constexpr bool MX = F == F_MX4 || F == F_MX8;
  constexpr int FS = F == F_F32 ? F_F32 : F_BF16;
  hipError_t err;
  const int pairs = a.T * a.k;
  const int quant = MX ? (a.T * a.d / 32 + 255) / 256 : 0;
  if (a.score_items + quant > 0) {
    hipLaunchKernelGGL((few_scores<FS>), dim3(a.score_items + quant), dim3(256), 0, s, a);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  const int shared = a.has_shared ? (a.I + 15) / 16 : 0;
  // lanes hold ceil(E / 64) experts: their selection takes groups of whole lanes,
  // a power of two of them
  const int size = a.E / a.G, epl = (a.E + 63) / 64, lanes = size / epl;
  const bool odd = a.route_mode == MOE_ROUTE_LEARNED && a.G > 1 &&
                   (size % epl != 0 || (lanes & (lanes - 1)) != 0);
  if (odd)
    hipLaunchKernelGGL((few_plan<FS, TILED && F != F_F32, true>), dim3(1 + shared), dim3(1024), 0, s,
                       a);
  else
    hipLaunchKernelGGL((few_plan<FS, TILED && F != F_F32, false>), dim3(1 + shared), dim3(1024), 0,
                       s, a);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  const int64_t up = (int64_t)pairs * ((a.I + 31) / 32);
  hipLaunchKernelGGL((few_up<F, TILED>), dim3(up < kGroups ? (unsigned)up : kGroups), dim3(256), 0,
                     s, a);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  // one wave a tile where the scales of all its inputs fit a wave's share of LDS.
  // Four waves | one in us a layer, at 1, 2, 5 and 16 tokens of 64 experts: bf16
  // activations 5120x1536 46.5 | 46.9, 65.1 | 62.8, 102.8 | 96.6, 174 | 166; 1024x256
  // 23.7 | 24.5, 24.7 | 25.6, 27.2 | 27.8, 38.0 | 36.3; MXFP8 5120x1536 44.8 | 42.9, 62.3 |
  // 59.2, 96.9 | 90.4, 156 | 146: up to 1 us behind where there are few tiles, up to 11
  // ahead where there are many
  constexpr bool FP4 = is_fp4<F>();
  const bool one = FP4 && a.I <= 7 * 256;
  const int64_t blocks = (a.d + 63) / 64;
  const int64_t down = (pairs * blocks + (one ? 3 : 0)) / (one ? 4 : 1) + (a.has_shared ? blocks : 0);
  const dim3 dg(down < kGroups ? (unsigned)down : kGroups);
  constexpr bool P = F != F_F32;
  if (one && a.T <= 8)
    hipLaunchKernelGGL((few_down<F, TILED, P, FP4 ? 1 : 4>), dg, dim3(256), 0, s, a);
  else if (one)
    hipLaunchKernelGGL((few_down<F, TILED, false, FP4 ? 1 : 4>), dg, dim3(256), 0, s, a);
  else if (P && a.T <= 8)
    hipLaunchKernelGGL((few_down<F, TILED, P, 4>), dg, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((few_down<F, TILED, false, 4>), dg, dim3(256), 0, s, a);
  if ((err = hipGetLastError()) != hipSuccess) return err;
  const dim3 grid((unsigned)((a.d + 1023) / 1024), (unsigned)a.T);
  if (F == F_F32) hipLaunchKernelGGL((few_combine<float>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((few_combine<bf16>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Parts of the inputs of the gate logits: workgroups for half the GPU, each
// wave still with stages to load.
int few_logit_parts(int d, bool f32) {
  const int nst = (d + (f32 ? 15 : 63)) / (f32 ? 16 : 64), parts = nst / 8;
  return parts < 1 ? 1 : parts > kLogitParts ? kLogitParts : parts;
}

hipError_t launch_few(FewArgs a, const moe_config &cfg, hipStream_t s) {
  const bool tiled = cfg.weight_layout == MOE_LAYOUT_TILED;
  const bool learned = cfg.route_mode == MOE_ROUTE_LEARNED;
  // A gate of at most 32 KB in rows of at most 2 KB (two bursts of loads a wave) and
  // 64 experts (what LDS holds): the routing workgroup computes its logits itself in
  // place of a launch.  Launch | itself in us a layer, one and 16 tokens: 8 KB (fp32,
  // 16 experts of 128) 19.9 | 18.5 and 23.5 | 22.1; 32 KB (32 of 256) 22.1 | 20.8 and
  // 25.6 | 25.0, (64 of 128) 20.3 | 19.7 and 24.0 | 24.4; 64 KB (64 of 256) 22.1 | 21.8
  // and 25.8 | 27.0, (32 of 512) 25.0 | 25.3 and 29.1 | 30.3; bf16 within 0.5 of that.
  // MXFP8 layers need the launch for x's codes.
  const int64_t gate_row = (int64_t)a.d * (cfg.act_dtype == MOE_DTYPE_F32 ? 4 : 2);
  a.small_gate = learned && a.E <= 64 && !a.xq && gate_row <= 2048 && a.E * gate_row <= 32768;
  a.score_items = learned && !a.small_gate ? (a.E + 15) / 16 * a.KS : 0;
  if (cfg.act_dtype == MOE_DTYPE_F32) return run_few<F_F32, false>(a, s);
  if (cfg.expert_dtype == MOE_DTYPE_FP8_E4M3_B128) return run_few<F_MX8, true>(a, s);
  if (cfg.expert_dtype == MOE_DTYPE_BF16)
    return tiled ? run_few<F_BF16, true>(a, s) : run_few<F_BF16, false>(a, s);
  if (cfg.act_quant == MOE_ACT_QUANT_MXFP8)
    return tiled ? run_few<F_MX4, true>(a, s) : run_few<F_MX4, false>(a, s);
  return tiled ? run_few<F_FP4, true>(a, s) : run_few<F_FP4, false>(a, s);
}

}  // namespace moe
