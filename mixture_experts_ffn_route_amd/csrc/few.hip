// The MoE layer for a few tokens (1 .. 16): moe_forward_few.
//
//   y[t] = sum_j w[t,j] FFN_{idx[t,j]}(x[t]) + FFN_shared(x[t])
//
// At these sizes the layer is a stream of the chosen experts' weights: every
// weight is used by one or two tokens, so the time is (bytes of the distinct
// chosen experts) / (HBM rate) plus launches and the waits between dependent
// steps.  The form here has three launches and no permutation:
//   front    gate logits (partial sums over parts of the input dimension),
//            the shared expert's gate|up, MXFP8 codes of x: what needs x alone
//   up       every workgroup selects the experts of all tokens itself from the
//            logits (the selection is microseconds of work on kilobytes, less
//            than another launch), then streams gate|up: H = SwiGLU
//   down     y: a workgroup owns 16 output columns and runs through all chosen
//            experts and the shared one, so the weighted sum over experts ends
//            in its registers and no combine is needed
//
// The token is the MFMA row: a product covers 16 rows x 16 weight columns, row
// t is token t for every expert, and rows of tokens that did not choose the
// expert are read as zeros (buffer loads out of range, which fetch nothing)
// and left out of the sum.  16 padded rows cost MFMA issue slots only, which a
// weight stream has to spare (a 1 KB weight fragment arrives per ~100 cycles
// and CU at the HBM rate; its MFMA takes 16).
//
// All loads are raw buffer loads: an offset past the resource's size reads 0
// and moves no data, which covers the stages past the end of a wave's share,
// the columns past a matrix's last row and the absent tokens without branches.

#include <climits>

#include "gemm.h"
#include "few.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kRows = MOE_FEW_MAX_TOKENS;      // MFMA rows = tokens
constexpr uint32_t kOut = 0x80000000u;         // an offset no resource here reaches

// Weight formats of a product.
enum { F_F32, F_BF16, F_FP4, F_MX4, F_MX8 };

// Inputs of one stage (the unit of a wave's load ring).
template <int F> constexpr int stage_inputs() { return F == F_F32 ? 16 : F == F_BF16 ? 64 : 128; }

__device__ __forceinline__ rsrc_t resource(const void *p, int64_t bytes) {
  const uint32_t n = bytes < (int64_t)kOut ? (uint32_t)bytes : kOut;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, n, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
}
__device__ __forceinline__ u32x4 load16_nt(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2);
}
__device__ __forceinline__ u32x2 load8_nt(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 2);
}
__device__ __forceinline__ uint32_t load4(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
__device__ __forceinline__ uint32_t load1(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
}

// One lane's operands of a stage.  Lane l: r = l % 16 (weight column, or token
// row), q = l / 16.  Inputs of lane q within a stage, the same for both sides:
//   F32   4q .. 4q+3 (one 16x16x4 MFMA per element)
//   BF16  8q .. 8q+7 and 32+8q .. 32+8q+7 (two 16x16x32)
//   FP4   32q .. 32q+31, the span of one scale byte (four 16x16x32 on 8 each)
//   MX4   weights 32q .. ; tokens 16q .. 16q+15 and 64+16q .. (one 16x16x128)
//   MX8   both as MX4's tokens
template <int F> struct BReg {
  u32x4 v[F == F_BF16 || F == F_MX8 ? 2 : 1];
  uint32_t s;
};
template <int F, bool HILO> struct AReg {
  u32x4 v[(F == F_F32 ? 1 : F == F_FP4 ? 4 : 2) * (HILO ? 2 : 1)];
  uint32_t s;
};

// Weight columns n0 .. n0+15 of an [N, K] matrix (and its scales).
struct BSrc {
  rsrc_t r, rs;
};
template <int F>
__device__ __forceinline__ BSrc b_source(const void *mat, const uint8_t *sc, int N, int K, int n0) {
  BSrc b;
  const int cols = N - n0 < 16 ? N - n0 : 16;
  if constexpr (F == F_F32 || F == F_BF16) {
    constexpr int es = F == F_F32 ? 4 : 2;
    b.r = resource((const uint8_t *)mat + (int64_t)n0 * K * es, (int64_t)cols * K * es);
    b.rs = b.r;
  } else if constexpr (F == F_MX8) {
    b.r = resource((const uint8_t *)mat + (int64_t)n0 * K, (int64_t)cols * K);
    b.rs = resource(sc + (int64_t)(n0 / 128) * (K / 128), K / 128);
  } else {
    b.r = resource((const uint8_t *)mat + (int64_t)n0 * (K / 2), (int64_t)cols * (K / 2));
    b.rs = resource(sc + (int64_t)n0 * (K / 32), (int64_t)cols * (K / 32));
  }
  return b;
}

// Stage st of the 16 columns; `out` is 0, or kOut for a stage that is not there.
template <int F, bool TILED>
__device__ __forceinline__ void load_b(BReg<F> &b, const BSrc &src, int K, int lane, int st,
                                       uint32_t out) {
  const uint32_t r = lane & 15, q = lane >> 4;
  if constexpr (F == F_F32) {
    const int k0 = st * 16 + 4 * q;
    if (K % 4 == 0) {
      b.v[0] = load16(src.r, (k0 < K ? (r * K + k0) * 4 : kOut) | out);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b.v[0][i] = load4(src.r, (k0 + i < K ? (r * K + k0 + i) * 4 : kOut) | out);
    }
  } else if constexpr (F == F_BF16) {
    const uint32_t off = TILED ? (uint32_t)st * 2048 + lane * 16 : r * K * 2 + st * 128 + q * 16;
    b.v[0] = load16_nt(src.r, off | out);
    b.v[1] = load16_nt(src.r, (off + (TILED ? 1024 : 64)) | out);
  } else if constexpr (F == F_MX8) {
    const uint32_t off = (uint32_t)st * 2048 + lane * 16;
    b.v[0] = load16_nt(src.r, off | out);
    b.v[1] = load16_nt(src.r, (off + 1024) | out);
    b.s = load1(src.rs, (uint32_t)st | out);
  } else {
    // K is a multiple of 64: the last stage may hold two lane groups only
    const uint32_t here = (st * 128 + (int)q * 32 < K ? 0 : kOut) | out;
    if constexpr (TILED) {
      const uint32_t tile = 2 * st + (q >> 1);
      const uint32_t off = tile * 512 + ((2 * (q & 1)) * 16 + r) * 8;
      const u32x2 lo = load8_nt(src.r, off | here), hi = load8_nt(src.r, (off + 128) | here);
      b.v[0] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      b.s = load1(src.rs, (tile * 32 + r * 2 + (q & 1)) | here);
    } else {
      b.v[0] = load16_nt(src.r, (r * (K / 2) + st * 64 + q * 16) | here);
      b.s = load1(src.rs, (r * (K / 32) + st * 4 + q) | here);
    }
  }
}

// Token rows: `row` is the lane's row of a [*, K] matrix (x, or H with its
// second bf16 half, or MXFP8 codes with scales), `out` as above (also kOut for
// a token that is not there).
struct ASrc {
  rsrc_t r, r2;                                // r2: low halves (HILO) or scales (MX)
};
template <int F, bool HILO>
__device__ __forceinline__ void load_a(AReg<F, HILO> &a, const ASrc &src, int K, int lane, int row,
                                       int st, uint32_t out) {
  const uint32_t q = lane >> 4;
  if constexpr (F == F_F32) {
    const int k0 = st * 16 + 4 * q;
    if (K % 4 == 0) {
      a.v[0] = load16(src.r, (k0 < K ? ((uint32_t)row * K + k0) * 4 : kOut) | out);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a.v[0][i] = load4(src.r, (k0 + i < K ? ((uint32_t)row * K + k0 + i) * 4 : kOut) | out);
    }
  } else if constexpr (F == F_BF16) {
    const uint32_t off = ((uint32_t)row * K + st * 64 + q * 8) * 2;
    a.v[0] = load16(src.r, off | out);
    a.v[1] = load16(src.r, (off + 64) | out);
    if constexpr (HILO) {
      a.v[2] = load16(src.r2, off | out);
      a.v[3] = load16(src.r2, (off + 64) | out);
    }
  } else if constexpr (F == F_FP4) {
    const uint32_t here = (st * 128 + (int)q * 32 < K ? 0 : kOut) | out;
    const uint32_t off = ((uint32_t)row * K + st * 128 + q * 32) * 2;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      a.v[s] = load16(src.r, (off + 16 * s) | here);
      if constexpr (HILO) a.v[4 + s] = load16(src.r2, (off + 16 * s) | here);
    }
  } else {
    const uint32_t off = (uint32_t)row * K + st * 128 + q * 16;
    a.v[0] = load16(src.r, off | out);
    a.v[1] = load16(src.r, (off + 64) | out);
    a.s = load1(src.r2, ((uint32_t)row * (K / 32) + st * 4 + q) | out);
  }
}

// acc += tokens x columns over one stage.
template <int F, bool HILO>
__device__ __forceinline__ void stage_mma(f32x4 &acc, const AReg<F, HILO> &a, const BReg<F> &b) {
  if constexpr (F == F_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[0][i]),
                                                 __uint_as_float(b.v[0][i]), acc, 0, 0, 0);
  } else if constexpr (F == F_BF16) {
#pragma unroll
    for (int h = 0; h < (HILO ? 4 : 2); ++h)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v[h]),
                                                    __builtin_bit_cast(bf16x8, b.v[h & 1]), acc, 0,
                                                    0, 0);
  } else if constexpr (F == F_FP4) {
    const float scale = __uint_as_float(b.s << 23);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const unsigned w = b.v[0][s];
      const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
      const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
      const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
      const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
      const bf16x8 bv = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v[s]), bv, acc, 0,
                                                    0, 0);
      if constexpr (HILO)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v[4 + s]), bv,
                                                      acc, 0, 0, 0);
    }
  } else {
    const i32x8 av = {(int)a.v[0][0], (int)a.v[0][1], (int)a.v[0][2], (int)a.v[0][3],
                      (int)a.v[1][0], (int)a.v[1][1], (int)a.v[1][2], (int)a.v[1][3]};
    if constexpr (F == F_MX4) {
      const i32x8 bv = {(int)b.v[0][0], (int)b.v[0][1], (int)b.v[0][2], (int)b.v[0][3], 0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 0, 4, 0, (int)a.s, 0,
                                                             (int)b.s);
    } else {
      const i32x8 bv = {(int)b.v[0][0], (int)b.v[0][1], (int)b.v[0][2], (int)b.v[0][3],
                        (int)b.v[1][0], (int)b.v[1][1], (int)b.v[1][2], (int)b.v[1][3]};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 0, 0, 0, (int)a.s, 0,
                                                             (int)b.s);
    }
  }
}

// A wave's share -- stages first, first + step, ... below end -- of the product
// of the token rows (those in `mask`) with 16 columns of NB matrices, DEPTH
// stages of loads in flight.
template <int F, int NB, bool TILED, int DEPTH>
__device__ __forceinline__ void rows_dot(f32x4 (&acc)[NB], const ASrc &as, const BSrc (&bs)[NB],
                                         int K, int lane, uint32_t mask, int first, int step,
                                         int end) {
  AReg<F, false> a[DEPTH];
  BReg<F> b[DEPTH][NB];
  const int row = lane & 15;
  const uint32_t absent = (mask >> row) & 1u ? 0u : kOut;
  auto load = [&](int p, int st) {
    const uint32_t out = st < end ? 0u : kOut;
#pragma unroll
    for (int n = 0; n < NB; ++n) load_b<F, TILED>(b[p][n], bs[n], K, lane, st, out);
    load_a<F, false>(a[p], as, K, lane, row, st, out | absent);
  };
#pragma unroll
  for (int p = 0; p < DEPTH; ++p) load(p, first + p * step);
  for (int st = first; st < end; st += DEPTH * step) {
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) {
#pragma unroll
      for (int n = 0; n < NB; ++n) stage_mma<F, false>(acc[n], a[p], b[p][n]);
      load(p, st + (p + DEPTH) * step);
    }
  }
}

// Sum of the waves' 16 x 16 partial products through LDS: element e = 16 row +
// column of matrix n, over waves w0 .. w0+count-1.
template <int NB>
__device__ __forceinline__ void put_partial(float *red, const f32x4 (&acc)[NB], int wave, int lane) {
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[(wave * NB + n) * 256 + ((lane >> 4) * 4 + i) * 16 + (lane & 15)] = acc[n][i];
}
template <int NB>
__device__ __forceinline__ float get_sum(const float *red, int n, int e, int w0, int count) {
  float v = 0.f;
  for (int w = w0; w < w0 + count; ++w) v += red[(w * NB + n) * 256 + e];
  return v;
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

// Shared exponent of an MXFP8 block with maximum magnitude amax (OCP MX).
__device__ __forceinline__ int mx_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int ex;
  frexpf(amax, &ex);
  const int X = ex - 1 - 8;
  return X < -127 ? -127 : (X > 127 ? 127 : X);
}
__device__ __forceinline__ float mx_element(float v, int X) {
  return fminf(fmaxf(ldexpf(v, -X), -448.f), 448.f);
}

// ---------------------------------------------------------------------------
// front: everything that needs x alone.  Blocks: gate logits (16 experts x one
// of KS parts of the input dimension), then 16 columns of the shared expert's
// gate|up, then blocks of 32 x values to MXFP8.
template <int F, bool TILED>
__global__ __launch_bounds__(512) void few_front(const FewArgs a) {
  __shared__ float red[8 * 2 * 256];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d = a.d, T = a.T;
  constexpr int es = F == F_F32 ? 4 : 2;
  constexpr int KST = stage_inputs<F>();
  const uint32_t all = (1u << T) - 1;
  const ASrc xs = {resource(a.x, (int64_t)T * d * es), resource(a.x, 0)};
  const int nst = (d + KST - 1) / KST;
  int item = blockIdx.x;
  if (item < a.logit_items) {
    const int part = item % a.KS, n0 = item / a.KS * 16;
    const int lo = (int)((int64_t)nst * part / a.KS), hi = (int)((int64_t)nst * (part + 1) / a.KS);
    const BSrc bs[1] = {b_source<F>(a.gate_w, nullptr, a.E, d, n0)};
    f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
    rows_dot<F, 1, false, 4>(acc, xs, bs, d, lane, all, lo + wave, waves, hi);
    put_partial<1>(red, acc, wave, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += blockDim.x) {
      const int t = e >> 4, n = n0 + (e & 15);
      if (t < T && n < a.E)
        a.zpart[((int64_t)part * T + t) * a.E + n] = get_sum<1>(red, 0, e, 0, waves);
    }
    return;
  }
  item -= a.logit_items;
  if (item < a.shared_items) {
    const int n0 = item * 16;
    const BSrc bs[2] = {b_source<F>(a.sh_gate, nullptr, a.I, d, n0),
                        b_source<F>(a.sh_up, nullptr, a.I, d, n0)};
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    rows_dot<F, 2, TILED, 4>(acc, xs, bs, d, lane, all, wave, waves, nst);
    put_partial<2>(red, acc, wave, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += blockDim.x) {
      const int t = e >> 4, n = n0 + (e & 15);
      if (t >= T || n >= a.I) continue;
      const float v = swiglu_pair(get_sum<2>(red, 0, e, 0, waves), get_sum<2>(red, 1, e, 0, waves),
                                  a.limit);
      const int64_t at = (int64_t)(T * a.k + t) * a.I + n;
      if constexpr (F == F_F32) ((float *)a.h)[at] = v;
      else store_hilo((bf16 *)a.h, (bf16 *)a.h_lo, at, v);
    }
    return;
  }
  item -= a.shared_items;
  if constexpr (F == F_BF16) {
    const int i = item * (int)blockDim.x + (int)threadIdx.x;
    if (!a.xq || i >= T * d / 32) return;
    const bf16 *p = (const bf16 *)a.x + (int64_t)i * 32;
    float v[32], amax = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = (float)p[j];
      amax = fmaxf(amax, fabsf(v[j]));
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
// affinities, bias, group limit, top-k and ties.  Lane l holds experts
// l*epl .. l*epl+epl-1.
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

__device__ __forceinline__ void select_few(const FewArgs &a, int t, int lane, float *out_w,
                                           int32_t *out_e) {
  constexpr int EPL = 8;                       // 512 experts at most
  const int E = a.E, epl = (E + 63) / 64;
  float s[EPL], key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    s[j] = -INFINITY;
    if (j < epl) {
      const int e = lane * epl + j;
      if (e < E) {
        float z = 0.f;
        for (int p = 0; p < a.KS; ++p) z += a.zpart[((int64_t)p * a.T + t) * E + e];
        s[j] = z;
      }
    }
  }
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, s[j]);
    m = wave_max(m);
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      s[j] = (j < epl && lane * epl + j < E) ? expf(s[j] - m) : 0.f;
      part += s[j];
    }
    const float inv = 1.f / wave_sum(part);
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] *= inv;
  } else if (a.score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j < epl) s[j] = 1.f / (1.f + expf(-s[j]));
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j < epl) s[j] = sqrtf(fmaxf(s[j], 0.f) + log1pf(expf(-fabsf(s[j]))));
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane * epl + j;
    key[j] = -INFINITY;
    if (j < epl && e < E) key[j] = a.bias ? s[j] + a.bias[e] : s[j];
    if (key[j] != key[j]) key[j] = -INFINITY;  // NaN scores come last
  }
  if (a.G > 1) {
    const int lpg = (E / a.G) / epl;           // a power of two (checked on the host)
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
    const float gs = a.bias ? (a1 + a2) : a1;
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
    float bv = -INFINITY;
    int bj = -1;                               // the lane's best untaken slot, lowest first
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j < epl && lane * epl + j < E && !((taken >> j) & 1u) && (bj < 0 || key[j] > bv)) {
        bv = key[j];
        bj = j;
      }
    const float m = wave_max_dpp(bv);
    // k <= E: some lane has an untaken expert at the maximum; lowest lane = lowest id
    const uint64_t at = __ballot(bj >= 0 && bv == m);
    const int owner = __builtin_ctzll(at);
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j == bj) mine = s[j];
    const int slot = __builtin_amdgcn_readlane(bj, owner);
    const float sv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), owner));
    if (lane == owner) taken |= 1u << slot;
    if (lane == r) { my_e = owner * epl + slot; my_s = sv; }
    ssum += sv;
  }
  if (lane < a.k) {
    float w = my_s;
    if (a.renorm) w = w / ssum;
    out_e[t * a.k + lane] = my_e;
    out_w[t * a.k + lane] = w * a.route_scale;
  }
}

// ---------------------------------------------------------------------------
// The plan of a call, the same for every workgroup: the distinct chosen
// experts ("slots", by first appearance in (token, choice) order), for each
// slot and token the H row (the pair's number t*k + j; -1: not chosen) and the
// gate value (summed where a token has the expert twice).
struct Plan {
  float *w;                                    // LDS [slots][16]
  int32_t *expert;                             // LDS [slots]
  int16_t *row;                                // LDS [slots][16]
};
// LDS bytes of a plan with `slots` slots (pairs, or pairs + 1 with the shared
// expert's) and of what building it takes.
__host__ __device__ inline int plan_bytes(int slots) { return slots * (64 + 4 + 32); }

__device__ __forceinline__ Plan plan_at(uint8_t *lds, int slots) {
  Plan p;
  p.w = (float *)lds;
  p.expert = (int32_t *)(lds + slots * 64);
  p.row = (int16_t *)(lds + slots * 68);
  return p;
}

// Routes all tokens and builds the plan; returns the number of slots.
// lds_w / lds_e: [T*k] gate values and expert ids; lead: [E] scratch.
__device__ __forceinline__ int make_plan(const FewArgs &a, const Plan &p, float *lds_w,
                                         int32_t *lds_e, int32_t *lead, int32_t *misc) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int T = a.T, k = a.k, E = a.E, pairs = T * k;
  if (tid == 0) misc[0] = 0;
  __syncthreads();
  if (a.route_mode == MOE_ROUTE_LEARNED) {
    for (int t = wave; t < T; t += waves) select_few(a, t, lane, lds_w, lds_e);
  } else if (tid < pairs) {
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
    lds_e[tid] = e;
    lds_w[tid] = ok ? a.route_scale / (float)k : 0.f;
    const int bad = (ok ? 0 : (int)MOE_FLAG_TOKEN_ID_RANGE) |
                    (e >= 0 && e < E ? 0 : (int)MOE_FLAG_EXPERT_RANGE);
    if (bad) atomicOr(&misc[0], bad);
  }
  __syncthreads();
  const int e = tid < pairs ? lds_e[tid] : -1;
  const bool in = e >= 0 && e < E;             // a table may hold ids past E: dropped
  if (in) lead[e] = INT_MAX;
  __syncthreads();
  if (in) atomicMin(&lead[e], tid);
  __syncthreads();
  const bool first = in && lead[e] == tid;
  // number of earlier leaders: pairs <= 256 are in the first four waves
  const uint64_t vote = __ballot(first);
  if (lane == 0 && wave < 4) misc[1 + wave] = __popcll(vote);
  __syncthreads();
  int slot = __popcll(vote & ((1ull << lane) - 1));
  for (int w = 0; w < wave && w < 4; ++w) slot += misc[1 + w];
  int slots = 0;
  for (int w = 0; w < 4 && w < waves; ++w) slots += misc[1 + w];
  if (first) {
    lead[e] = slot;
    p.expert[slot] = e;
  }
  for (int i = tid; i < slots * kRows; i += blockDim.x) {
    p.w[i] = 0.f;
    p.row[i] = -1;
  }
  __syncthreads();
  if (in) {
    const int t = tid / k, j = tid - t * k;
    float w = 0.f;
    bool mine = true;                          // the token's first choice of this expert
    for (int i = 0; i < k; ++i)
      if (lds_e[t * k + i] == e) {
        if (i < j) mine = false;
        w += lds_w[t * k + i];
      }
    if (mine) {
      p.w[lead[e] * kRows + t] = w;
      p.row[lead[e] * kRows + t] = (int16_t)tid;
    }
  }
  __syncthreads();
  return slots;
}

// up: H of every (slot, token) pair.  CB = 2 for MXFP8 (a scale block is 32
// columns): the waves halve over the two 16-column blocks of an item.
template <int F, bool TILED>
__global__ __launch_bounds__(512) void few_up(const FewArgs a) {
  constexpr bool MX = F == F_MX4 || F == F_MX8;
  constexpr int CB = MX ? 2 : 1;
  constexpr int KST = stage_inputs<F>();
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = a.T, d = a.d, I = a.I, pairs = T * a.k;
  // LDS: partial products | plan | routing of the pairs | scratch
  float *red = (float *)lds;
  uint8_t *at = lds + waves * 2 * 256 * 4;
  const Plan plan = plan_at(at, pairs);
  at += plan_bytes(pairs);
  float *lds_w = (float *)at;
  int32_t *lds_e = (int32_t *)(at + pairs * 4);
  int32_t *misc = (int32_t *)(at + pairs * 8);
  int32_t *lead = misc + 8;
  const int slots = make_plan(a, plan, lds_w, lds_e, lead, misc);
  if (blockIdx.x == 0) {
    // the routing for the caller, the plan for the down launch
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
      a.out_w[i] = lds_w[i];
      a.out_e[i] = lds_e[i];
    }
    for (int i = threadIdx.x; i < slots; i += blockDim.x) a.plan_expert[i] = plan.expert[i];
    for (int i = threadIdx.x; i < slots * kRows; i += blockDim.x) {
      a.plan_w[i] = plan.w[i];
      a.plan_row[i] = plan.row[i];
    }
    if (threadIdx.x == 0) {
      a.plan_slots[0] = slots;
      a.flags[0] = (uint32_t)misc[0];
    }
  }
  const int blocks = (I + 16 * CB - 1) / (16 * CB);
  const int nst = (d + KST - 1) / KST;
  constexpr int es = F == F_F32 ? 4 : 2;
  ASrc xs;
  if constexpr (MX) {
    xs.r = resource(a.xq, (int64_t)T * d);
    xs.r2 = resource(a.xq_scales, (int64_t)T * (d / 32));
  } else {
    xs.r = resource(a.x, (int64_t)T * d * es);
    xs.r2 = xs.r;
  }
  const int wpb = waves / CB;                  // waves per column block
  const int cb = CB == 1 ? 0 : wave / wpb;
  for (int item = blockIdx.x; item < slots * blocks; item += gridDim.x) {
    const int slot = item / blocks;
    const int n0 = (item - slot * blocks) * 16 * CB + cb * 16;
    const int e = __builtin_amdgcn_readfirstlane(plan.expert[slot]);
    const uint32_t mask =
        (uint32_t)__ballot(lane < kRows && plan.row[slot * kRows + (lane & 15)] >= 0);
    BSrc bs[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t *mat = (const uint8_t *)(n ? a.w_up : a.w_gate);
      const uint8_t *sc = n ? a.s_up : a.s_gate;
      const int64_t per = (int64_t)I * d;
      if constexpr (F == F_F32 || F == F_BF16) mat += e * per * es;
      else if constexpr (F == F_MX8) { mat += e * per; sc += e * (per / 16384); }
      else { mat += e * (per / 2); sc += e * (per / 32); }
      const int nu = __builtin_amdgcn_readfirstlane(n0);
      bs[n] = b_source<F>(mat, sc, I, d, nu);
    }
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    rows_dot<F, 2, TILED, 4>(acc, xs, bs, d, lane, mask, wave % wpb, wpb, nst);
    put_partial<2>(red, acc, wave, lane);
    __syncthreads();
    if constexpr (!MX) {
      for (int el = threadIdx.x; el < 256; el += blockDim.x) {
        const int t = el >> 4, n = n0 + (el & 15);
        const int pair = plan.row[slot * kRows + t];
        if (pair < 0 || n >= I) continue;
        const float v = swiglu_pair(get_sum<2>(red, 0, el, 0, waves),
                                    get_sum<2>(red, 1, el, 0, waves), a.limit);
        const int64_t o = (int64_t)pair * I + n;
        if constexpr (F == F_F32) ((float *)a.h)[o] = v;
        else store_hilo((bf16 *)a.h, (bf16 *)a.h_lo, o, v);
      }
    } else {
      // 8 waves: thread = (token, column of 32); the 32 lanes of a token share
      // the block's scale
      const int t = threadIdx.x >> 5, c = threadIdx.x & 31;
      const int el = t * 16 + (c & 15), w0 = (c >> 4) * wpb;
      const float v = swiglu_pair(get_sum<2>(red, 0, el, w0, wpb), get_sum<2>(red, 1, el, w0, wpb),
                                  a.limit);
      float amax = fabsf(v);
      amax = fmaxf(amax, xor_lane<1>(amax));
      amax = fmaxf(amax, xor_lane<2>(amax));
      amax = fmaxf(amax, xor_lane<4>(amax));
      amax = fmaxf(amax, xor_lane<8>(amax));
      amax = fmaxf(amax, xor_lane<16>(amax));
      const int X = mx_exponent(amax);
      const int word = __builtin_amdgcn_cvt_pk_fp8_f32(mx_element(v, X), 0.f, 0, false);
      const int pair = plan.row[slot * kRows + t];
      if (pair >= 0) {
        const int c0 = (item - slot * blocks) * 32;
        a.hq[(int64_t)pair * I + c0 + c] = (uint8_t)word;
        if (c == 0) a.hq_scales[(int64_t)pair * (I / 32) + c0 / 32] = (uint8_t)(X + 127);
      }
    }
    __syncthreads();
  }
}

// One wave's share of 16 columns of the down products: (slot, stage) pairs
// numbered slot by slot, this wave's first, first + step, ... of them.  Each
// stage's 16 x 16 product is scaled by the slot's gate values (row = token)
// and added.
template <int F, bool TILED, bool HILO, int DEPTH>
__device__ __forceinline__ void down_dot(f32x4 &total, const FewArgs &a, const Plan &plan,
                                         const ASrc &hs, const void *w, const uint8_t *sc,
                                         bool shared, int slot0, int slot1, int n0, int lane,
                                         int first, int step) {
  constexpr int KST = stage_inputs<F>();
  const int K = a.I, N = a.d, q = lane >> 4;
  const int nst = (K + KST - 1) / KST;
  AReg<F, HILO> ar[DEPTH];
  BReg<F> br[DEPTH];
  int at_slot[DEPTH];
  int slot = slot0 + first / nst, st = first % nst;        // the next stage to load
  auto load = [&](int p) {
    const bool there = slot < slot1;
    const int sl = there ? slot : slot1 - 1;
    at_slot[p] = sl;
    const uint32_t out = there ? 0u : kOut;
    const int e = shared ? 0 : __builtin_amdgcn_readfirstlane(plan.expert[sl]);
    const int64_t per = (int64_t)N * K;
    const uint8_t *mat = (const uint8_t *)w;
    const uint8_t *scale = sc;
    if constexpr (F == F_F32) mat += e * per * 4;
    else if constexpr (F == F_BF16) mat += e * per * 2;
    else if constexpr (F == F_MX8) { mat += e * per; scale += e * (per / 16384); }
    else { mat += e * (per / 2); scale += e * (per / 32); }
    const BSrc bs = b_source<F>(mat, scale, N, K, n0);
    load_b<F, TILED>(br[p], bs, K, lane, st, out);
    const int row = plan.row[sl * kRows + (lane & 15)];
    load_a<F, HILO>(ar[p], hs, K, lane, row < 0 ? 0 : row, st, out | (row < 0 ? kOut : 0u));
    st += step;
    while (st >= nst) { st -= nst; ++slot; }
  };
#pragma unroll
  for (int p = 0; p < DEPTH; ++p) load(p);
  const int n = (slot1 - slot0) * nst;
  for (int i = first; i < n; i += DEPTH * step) {
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      stage_mma<F, HILO>(acc, ar[p], br[p]);
      const f32x4 gv = *(const f32x4 *)(plan.w + at_slot[p] * kRows + 4 * q);
      // a token without this expert adds nothing, whatever the weights hold
#pragma unroll
      for (int r = 0; r < 4; ++r) total[r] += gv[r] != 0.f ? gv[r] * acc[r] : 0.f;
      load(p);
    }
  }
}

// down: y, 16 columns per workgroup.
template <int F, bool TILED>
__global__ __launch_bounds__(512) void few_down(const FewArgs a) {
  constexpr bool MX = F == F_MX4 || F == F_MX8;
  constexpr bool F32 = F == F_F32;
  constexpr int FS = F32 ? F_F32 : F_BF16;     // the shared expert's format
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = a.T, pairs = T * a.k;
  const int n0 = blockIdx.x * 16;
  float *red = (float *)lds;
  const Plan plan = plan_at(lds + waves * 256 * 4, pairs + 1);
  const int slots = a.plan_slots[0];
  for (int i = threadIdx.x; i < slots; i += blockDim.x) plan.expert[i] = a.plan_expert[i];
  for (int i = threadIdx.x; i < slots * kRows; i += blockDim.x) {
    plan.w[i] = a.plan_w[i];
    plan.row[i] = a.plan_row[i];
  }
  if (threadIdx.x < kRows) {                   // the shared expert: every token, weight 1
    const int t = threadIdx.x;
    plan.w[slots * kRows + t] = t < T ? 1.f : 0.f;
    plan.row[slots * kRows + t] = (int16_t)(t < T ? pairs + t : -1);
  }
  __syncthreads();
  f32x4 total = {0.f, 0.f, 0.f, 0.f};
  const int64_t rows = pairs + (a.has_shared ? T : 0);
  const int64_t hbytes = rows * a.I * (F32 ? 4 : 2);
  const ASrc hs = {resource(a.h, hbytes), resource(F32 ? a.h : a.h_lo, hbytes)};
  if (slots > 0) {
    if constexpr (MX) {
      const ASrc qs = {resource(a.hq, (int64_t)pairs * a.I),
                       resource(a.hq_scales, (int64_t)pairs * (a.I / 32))};
      down_dot<F, TILED, false, 4>(total, a, plan, qs, a.w_down, a.s_down, false, 0, slots, n0,
                                   lane, wave, waves);
    } else {
      down_dot<F, TILED, !F32, F == F_FP4 ? 3 : 4>(total, a, plan, hs, a.w_down, a.s_down, false,
                                                   0, slots, n0, lane, wave, waves);
    }
  }
  if (a.has_shared)
    down_dot<FS, TILED && !F32, !F32, 4>(total, a, plan, hs, a.sh_down, nullptr, true, slots,
                                         slots + 1, n0, lane, wave, waves);
  const f32x4 acc[1] = {total};
  put_partial<1>(red, acc, wave, lane);
  __syncthreads();
  for (int e = threadIdx.x; e < 256; e += blockDim.x) {
    const int t = e >> 4, n = n0 + (e & 15);
    if (t >= T || n >= a.d) continue;
    const float v = get_sum<1>(red, 0, e, 0, waves);
    if constexpr (F32) ((float *)a.y)[(int64_t)t * a.d + n] = v;
    else ((bf16 *)a.y)[(int64_t)t * a.d + n] = (bf16)v;
  }
}

template <int F, bool TILED>
hipError_t run_few(FewArgs a, hipStream_t s) {
  constexpr bool MX = F == F_MX4 || F == F_MX8;
  constexpr int FS = F == F_F32 ? F_F32 : F_BF16;
  hipError_t err;
  const int pairs = a.T * a.k;
  const int quant = MX ? (a.T * a.d / 32 + 511) / 512 : 0;
  const int front = a.logit_items + a.shared_items + quant;
  if (front > 0) {
    hipLaunchKernelGGL((few_front<FS, TILED && F != F_F32>), dim3(front), dim3(512), 0, s, a);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  {
    const int waves = 8;
    const int items = pairs * ((a.I + (MX ? 31 : 15)) / (MX ? 32 : 16));
    const int grid = items < 512 ? items : 512;
    const int lds = waves * 2 * 256 * 4 + plan_bytes(pairs) + pairs * 8 + 32 + a.E * 4;
    hipLaunchKernelGGL((few_up<F, TILED>), dim3(grid), dim3(waves * 64), lds, s, a);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  const int waves = 8;
  const int lds = waves * 256 * 4 + plan_bytes(pairs + 1);
  hipLaunchKernelGGL((few_down<F, TILED>), dim3((a.d + 15) / 16), dim3(waves * 64), lds, s, a);
  return hipGetLastError();
}

}  // namespace

// Parts of the input dimension of the gate logits: enough workgroups that a
// CU's share of the gate matrix is a few KB (latency, not bandwidth, is what
// the logits take), each wave still with two stages.
int few_logit_parts(int E, int d, bool f32) {
  const int nst = (d + (f32 ? 15 : 63)) / (f32 ? 16 : 64);
  int parts = nst / 16;
  return parts < 1 ? 1 : parts > 4 ? 4 : parts;
}

hipError_t launch_few(FewArgs a, const moe_config &cfg, hipStream_t s) {
  const bool f32 = cfg.act_dtype == MOE_DTYPE_F32;
  const bool tiled = cfg.weight_layout == MOE_LAYOUT_TILED;
  a.logit_items = cfg.route_mode == MOE_ROUTE_LEARNED ? (a.E + 15) / 16 * a.KS : 0;
  a.shared_items = a.has_shared ? (a.I + 15) / 16 : 0;
  if (f32) return run_few<F_F32, false>(a, s);
  if (cfg.expert_dtype == MOE_DTYPE_FP8_E4M3_B128) return run_few<F_MX8, true>(a, s);
  if (cfg.expert_dtype == MOE_DTYPE_BF16)
    return tiled ? run_few<F_BF16, true>(a, s) : run_few<F_BF16, false>(a, s);
  if (cfg.act_quant == MOE_ACT_QUANT_MXFP8)
    return tiled ? run_few<F_MX4, true>(a, s) : run_few<F_MX4, false>(a, s);
  return tiled ? run_few<F_FP4, true>(a, s) : run_few<F_FP4, false>(a, s);
}

}  // namespace moe
