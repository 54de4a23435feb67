// C ABI of what trains the MoE layer: checks of the arguments before the launches
// of rows.hip, checkpoint.hip and grouped.hip.  See moe.h for the contracts.

#include <cmath>
#include <initializer_list>

#include "train.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int32_t kMostColumns = INT32_MAX - 31;  // rounded up to whole pieces and blocks: 31 bits

bool misaligned(const void *p, size_t n) { return (uintptr_t)p % n != 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
size_t size_of(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

struct Range {
  const void *p;
  size_t n;
};
bool meet(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.n && y < x + a.n;
}
// Whether an output shares memory with an input or with another output.
bool overlap(std::initializer_list<Range> out, std::initializer_list<Range> in) {
  for (auto o = out.begin(); o != out.end(); ++o) {
    for (const Range &i : in)
      if (meet(*o, i)) return true;
    for (auto p = out.begin(); p != o; ++p)
      if (meet(*o, *p)) return true;
  }
  return false;
}

// Sizes of the calls that move rows; of the configuration dim, k and act_dtype.
int check_rows(const moe_config *c, int64_t T, int64_t R, const int32_t *inverse,
               moe::RowsArgs *a) {
  if (!c || c->dim < 1 || c->n_activated_experts < 1) return MOE_ERR_INVALID_ARG;
  if (c->act_dtype != MOE_DTYPE_F32 && c->act_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (T < 0 || R < 0) return MOE_ERR_INVALID_ARG;
  if (c->n_activated_experts > 16 || T > INT32_MAX / c->n_activated_experts || R > INT32_MAX ||
      c->dim > kMostColumns)
    return MOE_ERR_UNSUPPORTED;
  *a = {};
  a->inverse = inverse;
  a->T = T; a->R = R;
  a->d = c->dim; a->k = c->n_activated_experts; a->dtype = c->act_dtype;
  if (T == 0) return MOE_OK;
  if (moe::rows_threads(*a) >= (int64_t)1 << 32) return MOE_ERR_UNSUPPORTED;
  if (!inverse || misaligned(inverse, 4)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
// The memory of these calls' tensors.
struct RowsMemory {
  size_t tokens, rows, pairs;  // bytes: [T, d], [R, d], [T, k] of 4 bytes
  size_t es;
  explicit RowsMemory(const moe::RowsArgs &a)
      : tokens(size_of(a.dtype) * a.T * a.d), rows(size_of(a.dtype) * a.R * a.d),
        pairs((size_t)4 * a.T * a.k), es(size_of(a.dtype)) {}
};

int check_checkpoint(const void *m, int32_t dtype, int64_t rows, int32_t cols, int64_t ld,
                     const uint8_t *codes, const uint8_t *scales, moe::CheckpointArgs *a) {
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (ld == 0) ld = cols;
  if (ld < cols) return MOE_ERR_INVALID_ARG;
  if (rows > INT32_MAX || ld > INT32_MAX || cols > kMostColumns) return MOE_ERR_UNSUPPORTED;
  *a = {};
  a->rows = rows; a->cols = cols; a->ld = ld; a->dtype = dtype;
  if (rows == 0) return MOE_OK;
  if (moe::checkpoint_threads(*a) >= (int64_t)1 << 32) return MOE_ERR_UNSUPPORTED;
  if (!m || !codes || !scales || misaligned(m, size_of(dtype))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
size_t matrix_bytes(const moe::CheckpointArgs &a) {
  return size_of(a.dtype) * ((a.rows - 1) * a.ld + a.cols);
}
Range codes_of(const moe::CheckpointArgs &a) { return {a.codes, (size_t)(a.rows * a.cols)}; }
Range scales_of(const moe::CheckpointArgs &a) { return {a.scales, (size_t)(a.rows * ((a.cols + 31) / 32))}; }

// Of the configuration: dim, n_routed_experts, moe_inter_dim, swiglu_limit and the
// types; the routing's members are not read.
int check_experts(const moe_config *c, int64_t rows, const moe_experts_saved *saved,
                  moe::ExpertsArgs *a) {
  if (!c || c->dim < 1 || c->n_routed_experts < 1 || c->moe_inter_dim < 1 || rows < 0)
    return MOE_ERR_INVALID_ARG;
  if (c->act_dtype != MOE_DTYPE_F32 && c->act_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(c->swiglu_limit >= 0.f) || std::isinf(c->swiglu_limit)) return MOE_ERR_INVALID_ARG;
  if (saved && (saved->kind < MOE_SAVE_NONE || saved->kind > MOE_SAVE_MXFP8))
    return MOE_ERR_INVALID_ARG;
  if (c->expert_dtype != c->act_dtype || c->weight_layout != MOE_LAYOUT_ROWS ||
      c->act_quant != MOE_ACT_QUANT_NONE)
    return MOE_ERR_UNSUPPORTED;
  const int piece = c->act_dtype == MOE_DTYPE_F32 ? 4 : 8;
  if (c->dim % piece || c->moe_inter_dim % piece) return MOE_ERR_UNSUPPORTED;
  // a tile's rows are addressed with 32-bit byte offsets
  if (c->n_routed_experts > 1024 || c->dim > MOE_LINEAR_MAX_LD ||
      c->moe_inter_dim > MOE_LINEAR_MAX_LD || rows > INT32_MAX - 1024)
    return MOE_ERR_UNSUPPORTED;
  if (saved && saved->kind == MOE_SAVE_MXFP8 && c->moe_inter_dim % 32) return MOE_ERR_UNSUPPORTED;
  *a = {};
  a->rows = rows;
  a->d = c->dim; a->I = c->moe_inter_dim; a->E = c->n_routed_experts;
  a->dtype = c->act_dtype; a->limit = c->swiglu_limit;
  if (saved) a->saved = *saved;
  return moe::experts_launchable(*a, true) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
int check_saved(const moe_experts_saved &s) {
  if (s.kind == MOE_SAVE_NONE) return MOE_OK;
  if (!s.gate || !s.up || misaligned(s.gate, 16) || misaligned(s.up, 16)) return MOE_ERR_INVALID_ARG;
  if (s.kind == MOE_SAVE_MXFP8 && (!s.gate_scales || !s.up_scales)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
// The memory of a call's tensors.
struct ExpertsMemory {
  size_t rows, weights, kept, scales;
  explicit ExpertsMemory(const moe::ExpertsArgs &a) {
    const size_t es = size_of(a.dtype);
    rows = es * a.rows * a.d;
    weights = es * a.E * a.d * a.I;
    const bool mx = a.saved.kind == MOE_SAVE_MXFP8;
    kept = a.saved.kind == MOE_SAVE_NONE ? 0 : (size_t)(mx ? 1 : 4) * a.rows * a.I;
    scales = mx ? (size_t)a.rows * (a.I / 32) : 0;
  }
};

}  // namespace

extern "C" {

int moe_dispatch(const moe_config *cfg, const void *x, const int32_t *inverse, int64_t T, int64_t R,
                 void *rows, void *stream) {
  moe::RowsArgs a;
  const int st = check_rows(cfg, T, R, inverse, &a);
  if (st != MOE_OK || T == 0 || R == 0) return st;
  const RowsMemory m(a);
  if (!x || !rows || misaligned(x, m.es) || misaligned(rows, m.es)) return MOE_ERR_INVALID_ARG;
  if (overlap({{rows, m.rows}}, {{x, m.tokens}, {inverse, m.pairs}})) return MOE_ERR_INVALID_ARG;
  a.tokens = x; a.out_rows = rows;
  return hip_status(moe::launch_dispatch(a, (hipStream_t)stream));
}

int moe_dispatch_backward(const moe_config *cfg, const void *drows, const int32_t *inverse, int64_t T,
                          int64_t R, void *dx, void *stream) {
  moe::RowsArgs a;
  const int st = check_rows(cfg, T, R, inverse, &a);
  if (st != MOE_OK || T == 0) return st;
  const RowsMemory m(a);
  if ((!drows && R > 0) || !dx || misaligned(drows, m.es) || misaligned(dx, m.es))
    return MOE_ERR_INVALID_ARG;
  if (overlap({{dx, m.tokens}}, {{drows, m.rows}, {inverse, m.pairs}})) return MOE_ERR_INVALID_ARG;
  a.rows = drows; a.out_tokens = dx;
  return hip_status(moe::launch_combine(a, (hipStream_t)stream));
}

int moe_combine(const moe_config *cfg, const void *rows, const int32_t *inverse, const float *weights,
                const void *add, int64_t T, int64_t R, void *y, void *stream) {
  moe::RowsArgs a;
  const int st = check_rows(cfg, T, R, inverse, &a);
  if (st != MOE_OK || T == 0) return st;
  const RowsMemory m(a);
  if ((!rows && R > 0) || !weights || !y || misaligned(rows, m.es) || misaligned(weights, 4) ||
      misaligned(add, m.es) || misaligned(y, m.es))
    return MOE_ERR_INVALID_ARG;
  if (overlap({{y, m.tokens}},
              {{rows, m.rows}, {inverse, m.pairs}, {weights, m.pairs}, {add, m.tokens}}))
    return MOE_ERR_INVALID_ARG;
  a.rows = rows; a.weights = weights; a.tokens = add; a.out_tokens = y;
  return hip_status(moe::launch_combine(a, (hipStream_t)stream));
}

int moe_combine_backward(const moe_config *cfg, const void *dy, const void *rows,
                         const int32_t *inverse, const float *weights, int64_t T, int64_t R,
                         void *drows, float *dweights, void *stream) {
  moe::RowsArgs a;
  const int st = check_rows(cfg, T, R, inverse, &a);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!drows && !dweights) return R > 0 ? MOE_ERR_INVALID_ARG : MOE_OK;   // drows is empty
  const RowsMemory m(a);
  if (!dy || misaligned(dy, m.es) || (drows && !weights) || (dweights && !rows && R > 0))
    return MOE_ERR_INVALID_ARG;
  if (misaligned(rows, m.es) || misaligned(weights, 4) || misaligned(drows, m.es) ||
      misaligned(dweights, 4))
    return MOE_ERR_INVALID_ARG;
  if (overlap({{drows, m.rows}, {dweights, m.pairs}},
              {{dy, m.tokens}, {rows, m.rows}, {inverse, m.pairs}, {weights, m.pairs}}))
    return MOE_ERR_INVALID_ARG;
  a.tokens = dy; a.rows = rows; a.weights = weights; a.out_rows = drows; a.dweights = dweights;
  return hip_status(moe::launch_combine_backward(a, (hipStream_t)stream));
}

int moe_checkpoint_save(const void *src, int32_t dtype, int64_t rows, int32_t cols, int64_t ld_src,
                        float limit, uint8_t *codes, uint8_t *scales, void *stream) {
  moe::CheckpointArgs a;
  const int st = check_checkpoint(src, dtype, rows, cols, ld_src, codes, scales, &a);
  if (st != MOE_OK) return st;
  if (!(limit >= 0.f) || std::isinf(limit)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  a.src = src; a.codes = codes; a.scales = scales; a.limit = limit;
  if (overlap({codes_of(a), scales_of(a)}, {{src, matrix_bytes(a)}})) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_checkpoint_save(a, (hipStream_t)stream));
}

int moe_checkpoint_load(const uint8_t *codes, const uint8_t *scales, int32_t dtype, int64_t rows,
                        int32_t cols, int64_t ld_dst, void *dst, void *stream) {
  moe::CheckpointArgs a;
  const int st = check_checkpoint(dst, dtype, rows, cols, ld_dst, codes, scales, &a);
  if (st != MOE_OK || rows == 0) return st;
  a.dst = dst; a.codes = const_cast<uint8_t *>(codes); a.scales = const_cast<uint8_t *>(scales);
  if (overlap({{dst, matrix_bytes(a)}}, {codes_of(a), scales_of(a)})) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_checkpoint_load(a, (hipStream_t)stream));
}

size_t moe_experts_workspace_size(const moe_config *cfg, int64_t rows, int32_t backward) {
  moe::ExpertsArgs a;
  if (check_experts(cfg, rows, nullptr, &a) != MOE_OK) return 0;
  const size_t n = moe::experts_space(rows, a.I, a.dtype, backward != 0).total;
  return n > kAlign ? n : kAlign;
}

int moe_experts(const moe_config *cfg, const moe_weights *w, const void *x, const int32_t *offsets,
                int64_t rows, void *y, const moe_experts_saved *saved, void *ws, size_t ws_bytes,
                void *stream) {
  moe::ExpertsArgs a;
  int st = check_experts(cfg, rows, saved, &a);
  if (st != MOE_OK) return st;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !y || !offsets || !w->w_gate || !w->w_up || !w->w_down) return MOE_ERR_INVALID_ARG;
  if ((st = check_saved(a.saved)) != MOE_OK) return st;
  if (misaligned(x, 16) || misaligned(y, 16) || misaligned(offsets, 4) || misaligned(w->w_gate, 16) ||
      misaligned(w->w_up, 16) || misaligned(w->w_down, 16))
    return MOE_ERR_INVALID_ARG;
  const ExpertsMemory m(a);
  const size_t need = moe::experts_space(rows, a.I, a.dtype, false).total;
  if (!ws || misaligned(ws, kAlign) || ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (overlap({{y, m.rows}, {a.saved.gate, m.kept}, {a.saved.up, m.kept},
               {a.saved.gate_scales, m.scales}, {a.saved.up_scales, m.scales}, {ws, need}},
              {{x, m.rows}, {offsets, (size_t)4 * (a.E + 1)}, {w->w_gate, m.weights},
               {w->w_up, m.weights}, {w->w_down, m.weights}}))
    return MOE_ERR_INVALID_ARG;
  a.x = x; a.offsets = offsets; a.y = y;
  a.w_gate = w->w_gate; a.w_up = w->w_up; a.w_down = w->w_down;
  return hip_status(moe::launch_experts(a, (char *)ws, (hipStream_t)stream));
}

int moe_experts_backward(const moe_config *cfg, const moe_weights *w, const void *x,
                         const int32_t *offsets, int64_t rows, const void *dy,
                         const moe_experts_saved *saved, const moe_experts_grads *g, void *ws,
                         size_t ws_bytes, void *stream) {
  moe::ExpertsArgs a;
  int st = check_experts(cfg, rows, saved, &a);
  if (st != MOE_OK) return st;
  if (!w || !g || !offsets || misaligned(offsets, 4)) return MOE_ERR_INVALID_ARG;
  if (!g->dx && !g->dw_gate && !g->dw_up && !g->dw_down)
    return rows > 0 ? MOE_ERR_INVALID_ARG : MOE_OK;                       // dx is empty
  const bool up = g->dw_gate || g->dw_up;
  if (rows > 0) {
    if (!saved || saved->kind == MOE_SAVE_NONE || !dy || !w->w_down) return MOE_ERR_INVALID_ARG;
    if ((st = check_saved(a.saved)) != MOE_OK) return st;
    if ((g->dx && (!w->w_gate || !w->w_up)) || (up && !x)) return MOE_ERR_INVALID_ARG;
  }
  for (const void *p : {x, dy, w->w_gate, w->w_up, w->w_down, (const void *)g->dx,
                        (const void *)g->dw_gate, (const void *)g->dw_up, (const void *)g->dw_down})
    if (misaligned(p, 16)) return MOE_ERR_INVALID_ARG;
  const ExpertsMemory m(a);
  const size_t need = moe::experts_space(rows, a.I, a.dtype, true).total;
  if (need > 0 && (!ws || misaligned(ws, kAlign) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (overlap({{g->dx, m.rows}, {g->dw_gate, m.weights}, {g->dw_up, m.weights},
               {g->dw_down, m.weights}, {ws, need}},
              {{x, m.rows}, {dy, m.rows}, {offsets, (size_t)4 * (a.E + 1)}, {w->w_gate, m.weights},
               {w->w_up, m.weights}, {w->w_down, m.weights}, {a.saved.gate, m.kept},
               {a.saved.up, m.kept}, {a.saved.gate_scales, m.scales},
               {a.saved.up_scales, m.scales}}))
    return MOE_ERR_INVALID_ARG;
  a.x = x; a.offsets = offsets; a.dy = dy;
  a.w_gate = w->w_gate; a.w_up = w->w_up; a.w_down = w->w_down;
  a.dx = g->dx; a.dw_gate = g->dw_gate; a.dw_up = g->dw_up; a.dw_down = g->dw_down;
  return hip_status(moe::launch_experts_backward(a, (char *)ws, (hipStream_t)stream));
}

int moe_experts_path(const moe_config *cfg, int64_t rows, int32_t product, moe_experts_path_info *info) {
  moe::ExpertsArgs a;
  const int st = check_experts(cfg, rows, nullptr, &a);
  if (st != MOE_OK) return st;
  if (!info || product < MOE_EXPERTS_UP || product > MOE_EXPERTS_DW) return MOE_ERR_INVALID_ARG;
  *info = moe::experts_path(a, product);
  return MOE_OK;
}

}  // extern "C"
