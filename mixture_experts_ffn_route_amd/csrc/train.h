// Launch interface of what trains the MoE layer: token rows to their experts and
// back (rows.hip), 8-bit checkpoints (checkpoint.hip), the experts' products on
// sorted rows and their gradient (grouped.hip).
#pragma once

#include "internal.h"

namespace moe {

// Token rows [T, d] and sorted rows [R, d]; inverse [T, k] the row of each pair
// (outside [0, R): none).
struct RowsArgs {
  const int32_t *inverse;
  const float *weights;        // [T, k] or null
  const void *tokens;          // dispatch: x; combine: add or null; its gradient: dy
  const void *rows;            // combine and its gradient
  void *out_tokens, *out_rows;
  float *dweights;
  int64_t T, R;
  int d, k, dtype;
};
hipError_t launch_dispatch(const RowsArgs &a, hipStream_t s);
hipError_t launch_combine(const RowsArgs &a, hipStream_t s);
hipError_t launch_combine_backward(const RowsArgs &a, hipStream_t s);
// Threads of the largest launch of these.
int64_t rows_threads(const RowsArgs &a);

struct CheckpointArgs {
  const void *src;             // save
  void *dst;                   // load
  uint8_t *codes, *scales;
  int64_t rows, ld;
  int cols, dtype;
  float limit;
};
hipError_t launch_checkpoint_save(const CheckpointArgs &a, hipStream_t s);
hipError_t launch_checkpoint_load(const CheckpointArgs &a, hipStream_t s);
int64_t checkpoint_threads(const CheckpointArgs &a);

struct ExpertsArgs {
  const void *x, *dy, *w_gate, *w_up, *w_down;
  const int32_t *offsets;      // [E + 1]
  void *y, *dx, *dw_gate, *dw_up, *dw_down;
  moe_experts_saved saved;     // kind MOE_SAVE_NONE: none
  int64_t rows;                // of x
  int d, I, E, dtype;
  float limit;
};
// Offsets in bytes from the workspace base.
struct ExpertsSpace {
  size_t total;
  size_t h;                    // SwiGLU rows [rows, I]
  size_t dz, du;               // backward: gradients of the gate and up products
};
ExpertsSpace experts_space(int64_t rows, int I, int dtype, bool backward);
// Whether the tiles of each launch can be counted, whatever the offsets hold.
bool experts_launchable(const ExpertsArgs &a, bool backward);
moe_experts_path_info experts_path(const ExpertsArgs &a, int product);
hipError_t launch_experts(const ExpertsArgs &a, char *ws, hipStream_t s);
hipError_t launch_experts_backward(const ExpertsArgs &a, char *ws, hipStream_t s);

}  // namespace moe
