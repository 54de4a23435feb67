/*
 * moe.h -- C ABI of the MI355X (gfx950) mixture-of-experts feed-forward layer.
 *
 * The library computes the forward pass of a DeepSeek-style MoE FFN layer, and has the
 * operators that train one (moe_dispatch, moe_experts, moe_combine and their gradients):
 *
 *   y[t] = cast( sum_j w[t,j] * FFN_{idx[t,j]}(x[t]) + FFN_shared(x[t]) )
 *   FFN(u) = W_down( SiLU(min(W_gate u, L)) * clamp(W_up u, -L, L) )
 *
 * Sources (pages, by title and section):
 *   - "DeepSeek-V3.2-Exp - Routing weights": excerpts "gate-init",
 *     "gate-forward" (learned gate) and "moe-forward" (dispatch loop).
 *   - "DeepSeek V4.1 - Add shared": the V4.1 MoE class (FP4 routed experts,
 *     swiglu_limit, shared expert added to every token, y cast to x's dtype).
 *   - "From One Giant FFN to 384 Tiny Experts": Ch.1 SwiGLU, Ch.4 routed +
 *     shared formula, Ch.6 selection-only bias, Ch.11.1 hash-routed layers,
 *     Ch.11.2 Sqrt(Softplus) affinity, Ch.11.4 SwiGLU clamp, Ch.11.6 FP4.
 *   - "How was DeepSeek V4's tid2eid derived?": eq. (1)-(2) and the greedy
 *     least-loaded table construction.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless marked (host).  The caller owns
 *     every buffer; the library never allocates or frees device memory.
 *   - GPU work is enqueued on `stream` (a hipStream_t; NULL = the default
 *     stream) and the call returns without synchronising.  Outputs are
 *     valid once the stream reaches that point.
 *   - Arguments are validated on the host before any launch; invalid ones
 *     return MOE_ERR_INVALID_ARG (or MOE_ERR_UNSUPPORTED for valid-but-not-
 *     implemented shapes) and enqueue nothing.  A failed launch returns
 *     MOE_ERR_HIP.  No C++ exception crosses the ABI.
 *   - Weight matrices are [out, in] row-major with the input (K) dimension
 *     contiguous, like nn.Linear: gate weight [E, dim]; routed W_gate and
 *     W_up [E, I, dim]; W_down [E, dim, I]; shared [I, dim], [I, dim], [dim, I].
 *     Routed and shared expert matrices (and FP4 scales) may instead be
 *     given in the tiled layout that moe_pack_weights writes
 *     (moe_config.weight_layout = MOE_LAYOUT_TILED); same sizes, same values.
 *   - bf16 is IEEE-style bfloat16 (upper half of an fp32); fp32 is IEEE.
 *   - FP4 routed experts (MOE_DTYPE_FP4_E2M1): E2M1 codes packed two per
 *     byte along the input dimension, element 2i in the low nibble; one
 *     E8M0 scale byte (value 2^(e-127)) per 32 consecutive input elements
 *     of each output row (OCP MXFP4, 1x32 sub-blocks).
 *   - All calls are thread-safe: the library holds no mutable global state.
 *     Calls that share a workspace must be ordered on one stream.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,   /* bad pointer, size or config field            */
  MOE_ERR_UNSUPPORTED = -2,   /* valid config this build does not implement    */
  MOE_ERR_WORKSPACE = -3,     /* workspace missing, misaligned or too small    */
  MOE_ERR_HIP = -4            /* a HIP launch or runtime call failed           */
} moe_status;

typedef enum {                /* affinity s = f(z) of the logits z             */
  MOE_SCORE_SOFTMAX = 0,      /* softmax over the E routed experts             */
  MOE_SCORE_SIGMOID = 1,      /* 1 / (1 + exp(-z))                             */
  MOE_SCORE_SQRTSOFTPLUS = 2  /* sqrt(log(1 + exp(z)))                         */
} moe_score_func;

typedef enum {
  MOE_ROUTE_LEARNED = 0,      /* gate GEMM + affinity + bias + group top-k     */
  MOE_ROUTE_HASH = 1,         /* indices = tid2eid[token_id]                   */
  MOE_ROUTE_NGRAM_HASH = 2    /* 2-gram hash: token_ids holds [T, 2] pairs
                                 (previous id, current id); see moe_route     */
} moe_route_mode;

typedef enum {
  MOE_DTYPE_F32 = 0,
  MOE_DTYPE_BF16 = 1,
  MOE_DTYPE_FP4_E2M1 = 2,     /* routed experts only; see conventions above    */
  MOE_DTYPE_FP8_E4M3_B128 = 3 /* routed experts only: E4M3 codes in the layout
                                 moe_redequant_fp8 writes, one E8M0 scale per
                                 128 x 128 block (moe_weights.s_gate/s_up/s_down
                                 point to the [E, out/128, in/128] scales);
                                 needs act_quant MXFP8 and weight_layout TILED */
} moe_dtype;

typedef enum {
  MOE_LAYOUT_ROWS = 0,        /* expert matrices [out, in] row-major           */
  MOE_LAYOUT_TILED = 1        /* expert matrices as written by moe_pack_weights */
} moe_weight_layout;

typedef enum {
  MOE_ACT_QUANT_NONE = 0,     /* routed experts see the bf16 activations       */
  MOE_ACT_QUANT_MXFP8 = 1     /* FP4 routed experts: the activations entering
                                 each routed GEMM (gathered x; SwiGLU output H)
                                 are quantised to OCP MXFP8 (E4M3 + one E8M0
                                 scale per 32 inputs, shared exponent
                                 floor(log2 amax) - 8, nearest value, ties to
                                 even, saturating at 448) and multiplied with
                                 the stored FP4 codes on the scaled MFMA; needs
                                 expert_dtype FP4_E2M1, act_dtype BF16,
                                 dim % 128 == 0, moe_inter_dim % 128 == 0.  The
                                 shared expert keeps bf16 activations.  The
                                 FP8 computation of FP4 experts: "From One
                                 Giant FFN to 384 Tiny Experts", Ch.11.6.      */
} moe_act_quant;

/* Layer configuration.  Field names follow the model arguments of the
 * "gate-init" excerpt and the V4.1 MoE class. */
typedef struct {
  int32_t dim;                 /* model width d                                  */
  int32_t n_routed_experts;    /* E (1..1024; learned routing: 1..512)           */
  int32_t n_activated_experts; /* k experts per token (1..16, k <= E)            */
  int32_t n_expert_groups;     /* G (1 = no groups); E % G == 0                  */
  int32_t n_limited_groups;    /* groups kept per token, 1..G                    */
  int32_t moe_inter_dim;       /* expert intermediate width I (also the shared) */
  int32_t n_shared_experts;    /* 0 or 1                                         */
  int32_t score_func;          /* moe_score_func                                 */
  float route_scale;           /* weights are multiplied by this                 */
  int32_t renormalize;         /* -1: renormalise iff score_func != softmax; 0/1 */
  float swiglu_limit;          /* L > 0 clamps; 0 = no clamp                     */
  int32_t route_mode;          /* moe_route_mode                                 */
  int64_t vocab_size;          /* hash routing: rows of tid2eid; 2-gram hash:
                                  the vocabulary size m (1 .. 2^31 - 1)          */
  int32_t act_dtype;           /* x, y, gate weight, shared expert: F32 or BF16  */
  int32_t expert_dtype;        /* routed experts: F32 (act F32), BF16 or
                                  FP4_E2M1 (act BF16)                            */
  int32_t weight_layout;       /* moe_weight_layout of the routed and shared
                                  expert matrices; TILED needs act_dtype BF16    */
  int32_t act_quant;           /* moe_act_quant for the routed FP4 experts       */
} moe_config;

/* Layer weights; unused members may be NULL. */
typedef struct {
  const void *gate_w;          /* [E, dim] act_dtype (learned routing)           */
  const float *gate_bias;      /* [E] fp32 selection bias, or NULL               */
  const void *w_gate;          /* [E, I, dim] (FP4: bytes [E, I, dim/2])         */
  const void *w_up;            /* [E, I, dim] (FP4: bytes [E, I, dim/2])         */
  const void *w_down;          /* [E, dim, I] (FP4: bytes [E, dim, I/2])         */
  const uint8_t *s_gate;       /* FP4 only: E8M0 [E, I, dim/32]                  */
  const uint8_t *s_up;         /* FP4 only: E8M0 [E, I, dim/32]                  */
  const uint8_t *s_down;       /* FP4 only: E8M0 [E, dim, I/32]                  */
  const void *sh_gate;         /* shared expert [I, dim] act_dtype               */
  const void *sh_up;           /* shared expert [I, dim] act_dtype               */
  const void *sh_down;         /* shared expert [dim, I] act_dtype               */
  const int32_t *tid2eid;      /* hash routing: [vocab_size, k] expert ids       */
} moe_weights;

/* Byte offsets of the sub-buffers moe_forward keeps in its workspace.
 * Every offset is 256-byte aligned; the workspace base must be too. */
typedef struct {
  size_t total_bytes;
  size_t route_weights;        /* float [T, k]   gate values                     */
  size_t route_indices;        /* int32 [T, k]   expert ids                      */
  size_t counts;               /* int32 [E]      pairs per expert                */
  size_t offsets;              /* int32 [E + 1]  exclusive scan of counts        */
  size_t sorted_tok;           /* int32 [T*k + T] token of each permuted row;
                                  rows T*k.. are the shared expert's (row-T*k)   */
  size_t sorted_slot;          /* int32 [T*k]    slot of each permuted row       */
  size_t sorted_weight;        /* float [T*k]    gate value of each permuted row */
  size_t inverse;              /* int32 [T, k]   permuted row of pair (t, j)     */
  size_t tiles;                /* int32 [max_tiles, 4] GEMM work list           */
  size_t tile_count;           /* int32 [1]      tiles written by the permute    */
  size_t flags;                /* uint32 [4]     device error flags (below)      */
  size_t route_logits;         /* float          partial gate logits (learned
                                  bf16 routing; 0 bytes otherwise)               */
  size_t perm_hist;            /* int32          per-chunk expert histograms and
                                  per-expert totals                          */
  size_t xq;                   /* uint8 [T, dim] MXFP8 codes of x (act_quant)   */
  size_t xq_scales;            /* uint8 [T, dim/32] their E8M0 scales            */
  size_t hq;                   /* uint8 [T*k, I] MXFP8 codes of H's routed rows  */
  size_t hq_scales;            /* uint8 [T*k, I/32]                              */
  size_t h;                    /* [T*k + T, I]   SwiGLU activations (bf16/f32);
                                  MXFP8 layers may leave the routed rows unwritten
                                  (the gate|up GEMM writes hq directly)          */
  size_t yrows;                /* [T*k + T, dim] weighted expert outputs         */
  int32_t max_tiles;
  int32_t tile_rows;           /* rows per GEMM tile chosen for this (cfg, T)    */
} moe_ws_layout;

/* Device error flag bits (flags[0]); a non-zero word means some output rows
 * were produced from substitute data as described. */
#define MOE_FLAG_TOKEN_ID_RANGE 1u  /* hash: a token id outside [0, vocab): the
                                       token used tid2eid row 0 with weight 0   */
#define MOE_FLAG_EXPERT_RANGE   2u  /* permute: an expert id outside [0, E):
                                       that pair was dropped (inverse = -1)     */

/* Human-readable name of a status code (static string). */
const char *moe_status_string(int status);

/* Host-only check of a configuration (no GPU needed).  Returns MOE_OK,
 * MOE_ERR_INVALID_ARG for inconsistent fields (E % G, k > E,
 * n_limited_groups > G, k > n_limited_groups * E / G, bad enums, ...) or
 * MOE_ERR_UNSUPPORTED for shapes this build does not implement (bf16/FP4
 * paths need dim % 64 == 0 and I % 64 == 0; group ranges whose size over
 * ceil(E/64) is not a power of two). */
int moe_validate_config(const moe_config *cfg);

/* Greedy hash-routing table ("How was DeepSeek V4's tid2eid derived?",
 * section "Mathematical formulation" and its reference implementation).
 * Tokens are taken by decreasing p (equal p: ascending id); each gets the k
 * experts of smallest current load (equal loads: ascending expert id), stored
 * in ascending (load, id) order, and each of those loads grows by p_i / k.
 *   p        (host) [m] token frequencies, any order, non-negative
 *   tid2eid  (host) [m, k] output, row = token id
 *   load     (host) [n] final normalised loads f, or NULL
 *   max_vio, min_vio (host) max(f) * n - 1 and min(f) * n - 1, or NULL
 * Pure host code, O(m * n); returns MOE_ERR_INVALID_ARG for m < 1, n < 1,
 * k < 1, k > n, NULL p/tid2eid or a negative/NaN p. */
int moe_build_tid2eid(const double *p, int64_t m, int32_t n, int32_t k,
                      int32_t *tid2eid, double *load,
                      double *max_vio, double *min_vio);

/* Rewrite the expert matrices into the tiled layout the grouped GEMMs
 * stream contiguously (a storage format only: the tiled matrices hold the same
 * values, and moe_forward gives bit-identical results with either layout).
 * Done once when the weights are loaded, not per forward call.
 *   src  expert matrices in MOE_LAYOUT_ROWS (cfg->weight_layout is ignored):
 *        w_gate, w_up, w_down, the FP4 scales and the shared matrices; NULL
 *        members are skipped.  gate_w, gate_bias and tid2eid are not touched.
 *   dst  caller-allocated buffers of the same byte sizes for every non-NULL
 *        src member (the pointers are written through; dst's struct itself is
 *        read-only), not overlapping src.
 * Layout, for a matrix [N, K] of one expert (K = input dim; N, K % 64 == 0):
 *   bf16: 16 x 32 tiles, tile (n/16, k/32) at element ((n/16)*(K/32) + k/32)*512;
 *         inside a tile, element (n, k) at (((k%32)/8)*16 + n%16)*8 + k%8 (one
 *         16-byte group per MFMA lane: 16 outputs x 8 consecutive inputs).
 *   FP4 codes (bytes [N, K/2]): 16 x 64-input tiles of 512 bytes, tile
 *         (n/16, kb/32) at byte ((n/16)*(K/64) + kb/32)*512 for byte column kb;
 *         inside, byte (n, kb) at (((kb%32)/8)*16 + n%16)*8 + kb%8.
 *   FP4 scales ([N, K/32]): 32-byte tiles, scale (n, j) at
 *         ((n/16)*(K/64) + j/2)*32 + (n%16)*2 + j%2.
 *   Experts follow each other as in the row layout (expert e at e*N*K elements).
 * Returns MOE_ERR_INVALID_ARG for a NULL cfg/src/dst, a NULL dst member whose
 * src member is set, or an fp32 layer; validation as moe_validate_config. */
int moe_pack_weights(const moe_config *cfg, const moe_weights *src,
                     const moe_weights *dst, void *stream);

/* FP4 -> FP8 re-dequantisation of expert weights ("From One Giant FFN to 384
 * Tiny Experts", Ch.11.6: FP4 weights in 1x32 sub-blocks dequantised to FP8
 * E4M3 in 128 x 128 blocks for computation, lossless while the sub-block
 * scale ratios stay within a bound).
 *   codes         n_mat consecutive FP4 matrices [N, K/2] bytes, row layout
 *                 (conventions above)
 *   scales        their E8M0 scales [N, K/32]
 *   fp8           out: E4M3 codes, n_mat x N x K bytes in the FP8 expert
 *                 layout: per matrix, 16-row block nb and 128-input stage st,
 *                 a 2 KB block at byte ((nb*(K/128) + st)*2048 whose byte
 *                 ((h*4 + q)*16 + c)*16 + i is the element of row 16nb + c,
 *                 input 128st + 64h + 16q + i
 *   block_scales  out: E8M0 [n_mat, N/128, K/128]: B = s_max - 6 floored at
 *                 0, s_max the largest scale among the block's 32-input
 *                 sub-blocks holding a nonzero code (127 if none)
 *   lossy         out: uint8 [n_mat, N/128, K/128], 1 where some element's
 *                 E4M3 code (the nearest value to e2m1 x 2^(s - B), ties to
 *                 even, saturating at 448) is not exactly its FP4 value --
 *                 exactly the blocks with a nonzero sub-block whose scale is
 *                 more than 2^14 below s_max -- else 0
 * Device pointers, enqueued on `stream` (hipStream_t or NULL).  N and K must
 * be positive multiples of 128 (MOE_ERR_UNSUPPORTED otherwise); NULL
 * pointers or n_mat < 0 give MOE_ERR_INVALID_ARG. */
int moe_redequant_fp8(const uint8_t *codes, const uint8_t *scales, int64_t n_mat, int32_t N,
                      int32_t K, uint8_t *fp8, uint8_t *block_scales, uint8_t *lossy,
                      void *stream);

/* Multi-start variant of moe_build_tid2eid (same page, "Reference
 * implementation": tokens taken in a random order instead of by decreasing
 * frequency; several runs; the table with the lowest max_vio is kept).
 *   orders      (host) [n_starts, m] int64: each row a permutation of
 *               0..m-1, the order one run takes the tokens in (the caller
 *               draws them, e.g. with its own seeded generator)
 *   best_start  (host) out: row of `orders` whose table is returned (equal
 *               max_vio keeps the earlier row), or NULL
 * Other arguments and tie rules as moe_build_tid2eid.  Returns
 * MOE_ERR_INVALID_ARG for n_starts < 1, a NULL `orders` or a row that is not
 * a permutation. */
int moe_build_tid2eid_multistart(const double *p, int64_t m, int32_t n, int32_t k,
                                 const int64_t *orders, int32_t n_starts, int32_t *tid2eid,
                                 double *load, double *max_vio, double *min_vio,
                                 int32_t *best_start);

/* Auxiliary-loss-free bias update ("From One Giant FFN to 384 Tiny Experts",
 * Ch.6 and 7.1), run once per training step after a forward pass:
 *   counts  [E] int32 pairs routed to each expert in the batch (the
 *           forward's workspace `counts`)
 *   T       tokens in the batch; the balanced level is T * k / E
 *   gamma   update speed (V3: 0.001)
 *   bias    [E] fp32 selection bias, updated in place: experts above the
 *           balanced level get bias - gamma, experts below it bias + gamma,
 *           experts exactly at it keep their bias (compared exactly as
 *           counts[e] * E against T * k; each step is one fp32 operation)
 *   stats   [4] double out, or NULL: mean load, population variance of the
 *           counts, max_vio = max(counts) * E / (T * k) - 1 and min_vio
 *           likewise (the balance measures of the tid2eid page and the
 *           load-variance table of the MaxText pull request "Load balancing
 *           changes for Deepseek v4")
 * Returns MOE_ERR_INVALID_ARG for a NULL cfg/counts/bias, T < 1 or a
 * non-finite gamma. */
int moe_update_bias(const moe_config *cfg, const int32_t *counts, int64_t T, float gamma,
                    float *bias, double *stats, void *stream);

/* Workspace needed by moe_forward for T tokens, and where each part lives.
 * Host-only; layout may be NULL.  Returns MOE_OK or a validation error. */
int moe_workspace_layout(const moe_config *cfg, int64_t T,
                         moe_ws_layout *layout);
size_t moe_workspace_size(const moe_config *cfg, int64_t T); /* 0 if invalid */

/* Routing ("gate-forward" excerpt; hash rule of Ch.11.1; the 2-gram hash
 * of "How was DeepSeek V4's tid2eid derived?", section "An extreme case").
 *   x         [T, dim] act_dtype (learned routing; may be NULL for hash)
 *   token_ids hash: [T] int32 token ids; 2-gram hash: [T, 2] int32 pairs
 *             (previous token id or -1 at a sequence start, current id);
 *             ignored for learned routing
 *   weights   [T, k] float out: gate values (hash: route_scale / k)
 *   indices   [T, k] int32 out: expert ids, in descending biased-score
 *             order; equal scores go to the lower expert id.  2-gram hash:
 *             expert j = (a * q_j + b) mod E for the pair (a, b), q_j the
 *             j-th smallest prime above vocab_size, a = vocab_size at a
 *             sequence start; the same expert may appear more than once.
 *             Ids outside [0, vocab_size) route like token 0 (2-gram: like
 *             the pair (vocab_size, 0)) with weight 0 and set
 *             MOE_FLAG_TOKEN_ID_RANGE in the forward's flags
 * Learned routing runs in one kernel: a workgroup owns 32 tokens and all E
 * experts, the score GEMM (bf16 MFMA, fp32 accumulation; fp32 FMAs for fp32
 * layers) leaves the logits in LDS, and the affinity, bias, group limit,
 * top-k and renormalisation run there; only weights and indices are written.
 * moe_forward, which has a workspace, routes with a split form instead (the
 * score GEMM split over the input dimension, its fp32 partial logits added
 * in order by the selection kernel): measured faster at every batch size,
 * see moe_forward.  Both forms select identically. */
int moe_route(const moe_config *cfg, const moe_weights *w, const void *x,
              const int32_t *token_ids, int64_t T,
              float *weights, int32_t *indices, void *stream);

/* Permutation by expert (the bincount / where loop of "moe-forward").
 *   indices     [T, k] int32 expert ids
 *   counts      [E]    out: pairs per expert
 *   offsets     [E+1]  out: exclusive scan, offsets[E] = pairs kept
 *   sorted_tok  [T*k]  out: token of each permuted row
 *   sorted_slot [T*k]  out: slot of each permuted row
 *   inverse     [T, k] out: permuted row of each pair (-1 if dropped)
 * Rows of one expert are in ascending (token, slot) order, so the result is
 * deterministic.  Ids outside [0, E) are dropped and flagged in `flags`
 * (uint32 [4], may be NULL; the caller zeroes it beforehand). */
int moe_permute(const moe_config *cfg, const int32_t *indices, int64_t T,
                int32_t *counts, int32_t *offsets, int32_t *sorted_tok,
                int32_t *sorted_slot, int32_t *inverse, uint32_t *flags,
                void *stream);

/* Full layer forward: route -> permute -> grouped GEMM1 (gate|up + SwiGLU,
 * clamp) -> grouped GEMM2 (down, times the gate value) -> combine with the
 * shared expert.  No host synchronisation inside.
 *   x   [T, dim] act_dtype;  token_ids [T] int32 (hash routing only)
 *   y   [T, dim] act_dtype out (may not alias x)
 *   ws  device workspace of at least moe_workspace_size(cfg, T) bytes,
 *       256-byte aligned; its sub-buffers (moe_ws_layout) hold the
 *       routing, permutation and intermediates of this call afterwards.
 * Learned bf16 routing inside the forward uses the split score GEMM: kp
 * partial [T, E] fp32 logit slices go to the workspace (route_logits) and the
 * selection kernel adds them in order.  That costs a round trip of
 * kp * T * E * 4 bytes (V3 prefill, T = 4096, E = 256, kp = 8: 33.6 MB each
 * way), but spreads the gate-weight stream over many workgroups: the route
 * stage takes 48 us there against 99 us for moe_route's one-kernel form
 * (23 against 90 us at T = 64), whose workgroups must each stream the whole
 * gate matrix.
 * Everything is enqueued on `stream`; nothing persists between calls.  The
 * call enqueues only kernels (and, in the variants below, event records and
 * waits): no host synchronisation, allocation or memset.  So it can be
 * captured in a HIP graph and replayed; a replay reads x, the weights and the
 * workspace at the addresses given at capture.
 * T == 0 is a no-op.  MOE_ERR_WORKSPACE if ws is NULL, misaligned or small. */
int moe_forward(const moe_config *cfg, const moe_weights *w, const void *x,
                const int32_t *token_ids, int64_t T, void *y,
                void *ws, size_t ws_bytes, void *stream);

/* moe_forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the workspace is a fixed device array inside the library, one per GPU,
 * MOE_NOALLOC_SCRATCH_BYTES (64 MiB) large and held until the process ends.
 * The caller still passes the inputs, the weights and y; arguments and
 * results are as moe_forward's.
 *   Returns MOE_ERR_WORKSPACE, before any launch, when moe_workspace_size(cfg,
 *   T) exceeds MOE_NOALLOC_SCRATCH_BYTES (V3 / V4.1-Flash shapes: decode
 *   batches of up to a few hundred tokens fit; large prefill batches do not),
 *   MOE_ERR_HIP if the array's device address cannot be obtained.
 * The call allocates nothing: the array's device address is taken once per
 * GPU (hipGetSymbolAddress, on the first call there).  Nothing in it needs to
 * start at zero (the kernels clear their flag words themselves).  Every call
 * on one GPU uses the same array and it keeps the last call's contents:
 * calls that overlap on one GPU (two streams, or two host threads without
 * ordering) race on it, so the caller orders them.  The workspace views of
 * moe_ws_layout are not exposed for this entry point. */
#define MOE_NOALLOC_SCRATCH_BYTES (64ull << 20)
int moe_forward_noalloc(const moe_config *cfg, const moe_weights *w, const void *x,
                        const int32_t *token_ids, int64_t T, void *y, void *stream);

/* moe_forward for a few tokens (T of 1 .. MOE_FEW_MAX_TOKENS): the decode step
 * of a handful of sequences.  The same layer, with every routing, expert type,
 * activation encoding and weight layout that moe_forward takes, run as a stream
 * of the chosen experts' weights without a permutation.  Results agree with
 * moe_forward's to rounding (this form rounds less: H is kept to 16 bits and the
 * weighted expert outputs are summed in fp32); the routing follows the same
 * rules.  A NaN passes the clamp, and in MXFP8 rows a NaN or an infinity is the
 * NaN code, so that a token's bad input or weight shows in its output
 * (moe_forward has the clamp's or the code's bound in its place).
 *   x, token_ids, y, w, stream  as moe_forward; x, y, the matrices and the FP4
 *       scales 16-byte aligned
 *   ws  device workspace of at least moe_few_workspace_size(cfg, T) bytes,
 *       256-byte aligned.  Nothing in it needs to start at any value; after the
 *       call it holds the routing and the device error flags at the offsets of
 *       moe_few_layout
 * Only kernels are enqueued: no allocation, memset or synchronisation, so the
 * call can be captured in a HIP graph.  Calls that share a workspace must be
 * ordered on one stream.  T == 0 is a no-op; T above MOE_FEW_MAX_TOKENS, or a
 * dim or moe_inter_dim above MOE_FEW_MAX_DIM, is MOE_ERR_UNSUPPORTED.  Groups
 * may have any size, also those that moe_forward refuses. */
#define MOE_FEW_MAX_TOKENS 16
#define MOE_FEW_MAX_DIM (1 << 20)
typedef struct {
  size_t total_bytes;
  size_t route_weights;        /* float [T, k]   gate values                     */
  size_t route_indices;        /* int32 [T, k]   expert ids                      */
  size_t flags;                /* uint32 [4]     device error flags; flags[0] as
                                  moe_forward's: an expert id outside [0, E)
                                  (MOE_FLAG_EXPERT_RANGE) adds nothing           */
  size_t scores;               /* float          partial gate logits             */
  size_t plan_slots;           /* int32 [1]      distinct chosen experts         */
  size_t plan_experts;         /* int32 [T*k]    their ids, by first appearance  */
  size_t plan_weights;         /* float [T*k, 16] gate value per (expert, token) */
  size_t plan_rows;            /* int16 [T*k, 16] its row of h, -1: not chosen   */
  size_t plan_masks;           /* int32 [T]      choices that hold a row         */
  size_t xq, xq_scales;        /* MXFP8 copy of x (act_quant)                    */
  size_t hq, hq_scales;        /* MXFP8 SwiGLU rows [T*k, I] (act_quant)         */
  size_t h, h_lo;              /* SwiGLU rows [T*k + T, I]: fp32, or the high and
                                  low bf16 whose sum is the value (T*k .. : the
                                  shared expert's; MXFP8 layers: those alone)    */
  size_t yrows;                /* float [T*k + T, d] weighted expert outputs     */
} moe_few_layout;
int moe_few_workspace_layout(const moe_config *cfg, int64_t T, moe_few_layout *layout);
size_t moe_few_workspace_size(const moe_config *cfg, int64_t T); /* 0 if invalid */
int moe_forward_few(const moe_config *cfg, const moe_weights *w, const void *x,
                    const int32_t *token_ids, int64_t T, void *y,
                    void *ws, size_t ws_bytes, void *stream);

/* Stages of moe_forward in launch order (for moe_forward_profiled). */
#define MOE_STAGE_ROUTE 0     /* router kernel (or hash gather)                  */
#define MOE_STAGE_PERMUTE 1   /* permute kernel                                 */
#define MOE_STAGE_GEMM1 2     /* gate|up grouped GEMM + SwiGLU (routed + shared;
                                 routed only with a side stream, moe_forward_ex) */
#define MOE_STAGE_GEMM2 3     /* down grouped GEMM x gate value                  */
#define MOE_STAGE_COMBINE 4   /* gather-combine into y                          */
#define MOE_STAGE_COUNT 5

/* moe_forward that also records a timing event on `stream` before each stage
 * and after the last one, so the caller can time every kernel of the call.
 *   events (host) [MOE_STAGE_COUNT + 1] hipEvent_t handles created by the
 *   caller (hipEventCreate); event i precedes stage i, event COUNT follows
 *   the combine.  Results are identical to moe_forward's.  A failed
 *   hipEventRecord returns MOE_ERR_HIP. */
int moe_forward_profiled(const moe_config *cfg, const moe_weights *w, const void *x,
                         const int32_t *token_ids, int64_t T, void *y,
                         void *ws, size_t ws_bytes, void **events, void *stream);

/* moe_forward with optional stage events (as moe_forward_profiled; NULL: none)
 * and an optional second stream of the caller, `side_stream` (NULL: none;
 * not `stream` itself), on the same device.  For FP4 / FP8 expert layers with
 * bf16 activations the work that needs x alone -- the MXFP8 copy of x and the
 * shared expert -- is enqueued on side_stream, forked from `stream` at the
 * start of the call, so it runs while the latency-bound routing and
 * permutation run on `stream` (the shared expert's output is added to the
 * routed sum and depends on x alone, "DeepSeek V4.1 - Add shared", formula
 * of Delta_ffn; the shared experts' work placed in the routing's idle time,
 * "From One Giant FFN to 384 Tiny Experts", Ch.5.1); `stream` waits for x's copy before
 * the routed up GEMM and joins side_stream before the combine, so all work of
 * the call is ordered before whatever the caller enqueues on `stream` next,
 * and side_stream gets nothing the next call's fork does not order after
 * this call.  The fork and join events (three per host thread and device)
 * are created on a thread's first such call and kept until the process
 * ends; nothing else persists.  The stage events then time the routed launches
 * only.  Results are bit-identical to moe_forward's (the same kernels in the
 * same order per output).  Other layers ignore side_stream. */
int moe_forward_ex(const moe_config *cfg, const moe_weights *w, const void *x,
                   const int32_t *token_ids, int64_t T, void *y,
                   void *ws, size_t ws_bytes, void **events, void *stream,
                   void *side_stream);

/* Dense products of the feed-forward layers that stand between MoE layers: a
 * linear layer with bias, activation and residual in one call, and its
 * gradient.  A dense SwiGLU layer is two of them, the gate|up product with
 * MOE_ACTIVATION_SWIGLU and the down product with the residual stream.
 *
 *   z = x W^T + bias                     (swiglu: also zu = x W_up^T + bias_up)
 *   y = cast(act(z) + residual)
 *
 * swiglu: act = SiLU(min(z, L)) * clamp(zu, -L, L) for limit L > 0, SiLU(z) zu
 * for limit 0 ("From One Giant FFN to 384 Tiny Experts", Ch.1 and 11.4). */
typedef enum {
  MOE_ACTIVATION_NONE = 0,
  MOE_ACTIVATION_RELU = 1,
  MOE_ACTIVATION_SILU = 2,
  MOE_ACTIVATION_GELU = 3,       /* z Phi(z), the exact form (erf)               */
  MOE_ACTIVATION_GELU_TANH = 4,  /* its tanh form                                */
  MOE_ACTIVATION_SWIGLU = 5      /* two products, see above                      */
} moe_activation;

typedef struct {
  int64_t rows;                /* M (0 .. 2^31 - 1)                              */
  int32_t in_dim;              /* K >= 1                                         */
  int32_t out_dim;             /* N >= 1                                         */
  int32_t dtype;               /* moe_dtype F32 or BF16, of every tensor         */
  int32_t activation;          /* moe_activation                                 */
  float limit;                 /* swiglu clamp L > 0; 0: none                    */
  int64_t ld_x;                /* row strides in elements, 0 = contiguous: x
                                  (>= K), y and dy (>= N), residual (>= N); up
                                  to MOE_LINEAR_MAX_LD                           */
  int64_t ld_y;
  int64_t ld_residual;
} moe_linear_config;
#define MOE_LINEAR_MAX_LD (1 << 20)

typedef struct {               /* contiguous, dtype                              */
  const void *w;               /* [N, K]                                         */
  const void *w_up;            /* [N, K] swiglu only, else NULL                  */
  const void *bias;            /* [N], or NULL                                   */
  const void *bias_up;         /* [N] swiglu only, or NULL                       */
} moe_linear_weights;

typedef struct {               /* contiguous except dx; NULL: not wanted         */
  void *dx;                    /* [M, K], stride ld_dx                           */
  void *dw, *dw_up;            /* [N, K]                                         */
  void *dbias, *dbias_up;      /* [N]                                            */
  int64_t ld_dx;               /* 0: K                                           */
} moe_linear_grads;

/* Workspace of moe_linear (backward = 0) or moe_linear_backward (backward = 1,
 * for every gradient).  Host-only; 0 for a configuration that the call refuses,
 * 256 at least for one that it takes. */
size_t moe_linear_workspace_size(const moe_linear_config *cfg, int32_t backward);

/* The forward product.
 *   x         [M, K] stride ld_x
 *   residual  [M, N] stride ld_residual, or NULL; may be y itself (same stride)
 *   y         [M, N] stride ld_y out
 *   z, z_up   [M, N] contiguous out, or NULL: the pre-activations z (and zu),
 *             which the gradient needs unless the activation is NONE.  Rounded
 *             to dtype, but never across the clamp's border
 *   ws        device workspace of at least moe_linear_workspace_size(cfg, 0)
 *             bytes, 256-byte aligned; nothing in it needs to start at any
 *             value.  Calls that share one must be ordered on one stream
 * Products accumulate in fp32, the epilogue is fp32, y is rounded once.  All
 * sizes and strides are taken; for large products, rows that are not whole
 * 16-byte pieces are first copied to padded ones in the workspace.  Alignment: x
 * and w, w_up 16 bytes where their rows are whole 16-byte pieces at 16-byte
 * strides, an element's size where not; the others an element's size.  No output
 * may overlap an input (but y the residual) or another output.  Results do not
 * depend on what else runs (no atomics).  Only kernels are enqueued on `stream`, so the call
 * can be captured in a HIP graph.  rows == 0 is a no-op.  Sizes whose launch
 * would have 2^32 threads or more (2^30 rows of 64 columns, or padded copies of
 * 2^32 16-byte pieces) are MOE_ERR_UNSUPPORTED. */
int moe_linear(const moe_linear_config *cfg, const moe_linear_weights *w, const void *x,
               const void *residual, void *y, void *z, void *z_up,
               void *ws, size_t ws_bytes, void *stream);

/* The gradient of moe_linear for the output gradient dy:
 *   dz = dy act'(z)          (swiglu: for both products; a clamped value has none)
 *   dx = dz W,  dW = dz^T x,  dbias = sum over rows of dz;  dresidual is dy
 *   dy        [M, N] stride ld_y, aligned as x and w are
 *   z, z_up   as moe_linear wrote them (activation NONE: ignored)
 *   x         needed for dw / dw_up; w->w, w->w_up for dx; else may be NULL
 *             (biases are not read)
 *   grads     at least one member; outputs are overwritten, not added to
 * Large products round dz to dtype first, as their matrix cores take it: with
 * the rounding of z that makes bf16 gradients 3e-3 of their norm off, where
 * fp32 throughout is 1.7e-3 off (the output's own rounding); small ones keep dz
 * in fp32.  Sums are fp32, outputs are rounded once.  No output may overlap an
 * input or another output.  rows == 0 writes zeros to the weight and bias
 * gradients. */
int moe_linear_backward(const moe_linear_config *cfg, const moe_linear_weights *w, const void *x,
                        const void *dy, const void *z, const void *z_up,
                        const moe_linear_grads *grads, void *ws, size_t ws_bytes, void *stream);

/* Which kernels a product of these calls takes (host-only, for tests and
 * profiles): a choice by sizes, types and row strides alone.  Of the backward
 * products, DX and DW; DW is both weight gradients of swiglu in one launch. */
typedef enum {
  MOE_LINEAR_FORWARD = 0,
  MOE_LINEAR_DX = 1,
  MOE_LINEAR_DW = 2
} moe_linear_product;
typedef enum {
  MOE_LINEAR_PATH_TILED = 0,   /* 64..256-square tiles, with copies of odd rows  */
  MOE_LINEAR_PATH_FEW = 1,     /* up to 16 rows: a stream of the weights         */
  MOE_LINEAR_PATH_SMALL = 2    /* 32 x 32 tiles, elements read one by one        */
} moe_linear_path_kind;
typedef struct {
  int32_t path;                /* moe_linear_path_kind                           */
  int32_t tile_rows;           /* tiled, else 0: a workgroup's rows and columns  */
  int32_t tile_cols;           /* (swiglu forward: columns of both products)     */
  int32_t parts;               /* workgroups that share a tile's contraction     */
} moe_linear_path_info;
int moe_linear_path(const moe_linear_config *cfg, int32_t product, moe_linear_path_info *info);

/* What trains the MoE layer: token rows to their experts and back with the gate
 * values, the experts' products on sorted rows, each with its gradient, and 8-bit
 * checkpoints of activations.  A training step of the routed experts is
 *   moe_route, moe_permute, moe_dispatch, moe_experts, moe_combine
 *   moe_combine_backward, moe_experts_backward, moe_dispatch_backward
 * with moe_dispatch again before moe_experts_backward where the sorted rows of x
 * were not kept (they are k times x).  "DeepSeek-V3.2-Exp - Routing weights",
 * excerpt "moe-forward", is the forward part.
 *
 * Token rows to their experts and back.  Of cfg: dim, n_activated_experts (k, 1 ..
 * 16) and act_dtype (F32 or BF16, of every row); any dim.
 *   inverse   [T, k] int32: the sorted row of each pair, as moe_permute writes it;
 *             one outside [0, R) has none (a dropped pair) and takes no part.  No
 *             row stands twice in it
 *   x, y, dx, dy, add  [T, dim];   rows, drows  [R, dim];   all contiguous
 *   weights, dweights  [T, k] float
 * Sums are fp32, over the slots in order; results are rounded once and do not
 * depend on what else runs.  Alignment: an element's size.  No output may overlap
 * an input or another output.  T == 0 is a no-op.  Sizes whose launch would have 2^32
 * threads (a thread takes 16 bytes of a token's row, and 2^24 tokens can have as many), or
 * with dim past 2^31 - 32, are MOE_ERR_UNSUPPORTED.  Only kernels are enqueued, so the
 * calls can be captured in a HIP graph.
 *
 * rows[inverse[t, j]] = x[t]; sorted rows that stand in no pair are left alone. */
int moe_dispatch(const moe_config *cfg, const void *x, const int32_t *inverse, int64_t T, int64_t R,
                 void *rows, void *stream);
/* dx[t] = sum over j of drows[inverse[t, j]]. */
int moe_dispatch_backward(const moe_config *cfg, const void *drows, const int32_t *inverse, int64_t T,
                          int64_t R, void *dx, void *stream);
/* y[t] = sum over j of weights[t, j] rows[inverse[t, j]], + add[t] (the shared
 * expert's output or a residual; NULL: none).  The gradient of add is that of y. */
int moe_combine(const moe_config *cfg, const void *rows, const int32_t *inverse, const float *weights,
                const void *add, int64_t T, int64_t R, void *y, void *stream);
/* drows[inverse[t, j]] = weights[t, j] dy[t] (other rows are left alone) and
 * dweights[t, j] = rows[inverse[t, j]] . dy[t] (0 where a pair has no row).  Either
 * may be NULL: not wanted (both: only where T or R is 0); rows is read for dweights
 * alone, weights for drows. */
int moe_combine_backward(const moe_config *cfg, const void *dy, const void *rows,
                         const int32_t *inverse, const float *weights, int64_t T, int64_t R,
                         void *drows, float *dweights, void *stream);

/* 8-bit checkpoints: a matrix kept in 1 + 1/32 bytes a value between the forward
 * and the backward pass (pre-activations of moe_linear, for one).  Per 32
 * consecutive columns of a row (fewer at its end) one E8M0 scale byte X + 127 and
 * E4M3 codes of v / 2^X, nearest value, ties to even; X is the least integer >= -127
 * with max|v| <= 448 2^X, 0 for a block of zeros: nothing saturates, a value is off
 * by 2^-4 of itself at most (below 2^-6 2^X: by 2^-10 2^X; at the top of the range see
 * below).
 * limit > 0: no value is carried across +-limit (the next code on the value's side
 * is taken), because the gradient of a clamp goes by the saved value; 0: no clamp.
 * NaN and infinities are kept as NaN and do not count for X.  Finite values from
 * 1.9375 2^127 on in magnitude, and those above a limit that is 1.875 2^127 or more, take
 * the code of 2^128 and come back as infinities of their sign.
 *   src, dst  [rows, cols] dtype (F32 or BF16), row stride ld elements (0: cols)
 *   codes     [rows, cols] bytes;   scales  [rows, ceil(cols / 32)] bytes
 * Any sizes (to 2^31 - 32 columns, and below 2^32 pieces of 16 bytes) and strides;
 * alignment an element's size.  Outputs may not overlap inputs.  rows == 0 is a
 * no-op. */
int moe_checkpoint_save(const void *src, int32_t dtype, int64_t rows, int32_t cols, int64_t ld_src,
                        float limit, uint8_t *codes, uint8_t *scales, void *stream);
int moe_checkpoint_load(const uint8_t *codes, const uint8_t *scales, int32_t dtype, int64_t rows,
                        int32_t cols, int64_t ld_dst, void *dst, void *stream);

/* The routed experts on sorted rows.  For the rows r of expert e, offsets[e] ..
 * offsets[e + 1]:
 *   z = x W_gate^T, u = x W_up^T, y = (SiLU(min(z, L)) clamp(u, -L, L)) W_down^T
 * without the gate value, which moe_combine applies.  Of cfg: dim,
 * n_routed_experts (E, or one rank's share; to 1024), moe_inter_dim (I),
 * swiglu_limit (L, 0: no clamp), act_dtype = expert_dtype (F32 or BF16),
 * weight_layout ROWS, act_quant NONE; dim and I whole 16-byte pieces (multiples of 8
 * in bf16, of 4 in fp32); other types, layouts and widths are MOE_ERR_UNSUPPORTED.
 *   w         w_gate, w_up [E, I, dim], w_down [E, dim, I]
 *   x, y      [rows, dim]; rows of no expert (rows >= offsets[E]: room that a batch
 *             leaves) are neither read nor written, here and in the gradient
 *   offsets   [E + 1] int32 on the device, as moe_permute writes it.  Values outside
 *             [0, rows] are clamped, and an expert that ends before it starts has no
 *             rows: no access is out of range, but rows that two experts then share
 *             have either's result (2^31 - 1024 rows and more, and sizes that could
 *             come near 2^31 tiles, are MOE_ERR_UNSUPPORTED)
 *   saved     where z and u go for the gradient: kind FULL in fp32, as they are; kind
 *             MXFP8 as moe_checkpoint_save with limit L keeps them, in a quarter of
 *             the memory (I % 32 == 0).  NULL or kind NONE: not saved
 *   ws        moe_experts_workspace_size(cfg, rows, 0) bytes, 256-byte aligned;
 *             nothing in it needs to start at any value.  Calls that share one must
 *             be ordered on one stream
 * Products accumulate in fp32; h = SiLU(..) clamp(..) is rounded to the type once
 * (as the next product takes it), y once.  Matrices 16-byte aligned.  No output may
 * overlap an input or another output.  Results do not depend on what else runs (no
 * atomics).  Only kernels are enqueued: the calls can be captured in a HIP graph,
 * whose replays may have other offsets.  rows == 0 is a no-op. */
typedef enum {
  MOE_SAVE_NONE = 0,
  MOE_SAVE_FULL = 1,
  MOE_SAVE_MXFP8 = 2
} moe_save_kind;
typedef struct {
  int32_t kind;                /* moe_save_kind                                  */
  void *gate, *up;             /* z, u: [rows, I] float, or bytes (codes)        */
  uint8_t *gate_scales;        /* MXFP8: [rows, I / 32]                          */
  uint8_t *up_scales;
} moe_experts_saved;
typedef struct {               /* NULL: not wanted; contiguous                   */
  void *dx;                    /* [rows, dim]                                    */
  void *dw_gate, *dw_up;       /* [E, I, dim]                                    */
  void *dw_down;               /* [E, dim, I]                                    */
} moe_experts_grads;
size_t moe_experts_workspace_size(const moe_config *cfg, int64_t rows, int32_t backward);
int moe_experts(const moe_config *cfg, const moe_weights *w, const void *x, const int32_t *offsets,
                int64_t rows, void *y, const moe_experts_saved *saved, void *ws, size_t ws_bytes,
                void *stream);
/* Its gradient for dy [rows, dim]:
 *   dh = dy W_down, dz = dh clamp(u) SiLU'(z) where z <= L, du = dh SiLU(z) where
 *   |u| <= L, both 0 elsewhere; h from z and u again
 *   dx = dz W_gate + du W_up, dw_gate = dz^T x, dw_up = du^T x, dw_down = dy^T h
 * with z and u as `saved` holds them.  Outputs are overwritten; an expert without
 * rows gets zeros.  w_down is always read, w_gate and w_up for dx, x for dw_gate and
 * dw_up; w's others may be NULL.  dz, du and h are rounded to the type once, as the
 * products take them.  ws: moe_experts_workspace_size(cfg, rows, 1) bytes.
 * rows == 0 writes zeros to the weight gradients that are wanted, and dx, empty, may be
 * NULL. */
int moe_experts_backward(const moe_config *cfg, const moe_weights *w, const void *x,
                         const int32_t *offsets, int64_t rows, const void *dy,
                         const moe_experts_saved *saved, const moe_experts_grads *grads, void *ws,
                         size_t ws_bytes, void *stream);

/* Tiles of the products of these calls (host-only, for tests and profiles): a choice by
 * sizes and types alone. */
typedef enum {
  MOE_EXPERTS_UP = 0,          /* z and u, h                                     */
  MOE_EXPERTS_DOWN = 1,        /* y                                              */
  MOE_EXPERTS_DH = 2,          /* dh; dz, du and h                               */
  MOE_EXPERTS_DX = 3,
  MOE_EXPERTS_DW_DOWN = 4,
  MOE_EXPERTS_DW = 5           /* dw_gate and dw_up                              */
} moe_experts_product;
typedef struct {
  int32_t tile_rows;           /* at most: lower ones for what is left           */
  int32_t tile_cols;           /* (UP: columns of both matrices)                 */
  int32_t streamed;            /* the weights pass the caches by                 */
} moe_experts_path_info;
int moe_experts_path(const moe_config *cfg, int64_t rows, int32_t product, moe_experts_path_info *info);

/* Roofline probes: the achievable HBM read rate and bf16 / FP8 MFMA rates of
 * the GPU, measured with the instruction forms the layer kernels use (16-byte
 * nontemporal vector loads; v_mfma_f32_16x16x32_bf16, v_mfma_f32_32x32x16_bf16,
 * v_mfma_scale_f32_16x16x128_f8f6f4), for the caller to time on `stream` and
 * report next to the data-sheet peaks.  Neither touches the layer state.
 *   moe_probe_read: reads `bytes` (a multiple of 16) of `buf` (16-byte
 *     aligned); 1024 workgroups of 4 waves, each wave streaming its own
 *     contiguous share with 1 KB loads, 8 in flight.  out: uint32 [1024]
 *     device scratch, written only if the loaded words hash to one fixed
 *     value (so the loads cannot be dropped).
 *   moe_probe_mfma: 2048 workgroups x 4 waves, each wave `iters` rounds of 8
 *     independent bf16 MFMAs, 16x16x32 (shape 0) or 32x32x16 (shape 1), or
 *     of 16 independent scaled 16x16x128 MFMAs on E4M3 x E2M1 (shape 2, the
 *     MXFP8 x MXFP4 expert GEMMs) or E4M3 x E4M3 (shape 3).
 *     out: float [2048] device scratch, written likewise; *flops (host)
 *     receives the flops the launch performs.
 * Return MOE_ERR_INVALID_ARG for NULL/misaligned pointers, bytes < 16,
 * iters < 1 or another shape. */
int moe_probe_read(const void *buf, int64_t bytes, void *out, void *stream);
int moe_probe_mfma(int32_t iters, int32_t shape, void *out, double *flops, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
