// Launch interface of the dense product (linear.hip): moe_linear and its
// gradient.
#pragma once

#include "internal.h"

namespace moe {

// Sizes and workspace of one moe_linear (or moe_linear_backward) call; offsets
// in bytes from the workspace base, 0-byte parts are not used.
struct LinearSpace {
  size_t total;
  size_t x, w, w_up;           // copies with 16-byte rows, where a row has none
  size_t dz, du;               // backward: gradient of the products' outputs
  size_t colsum;               // backward: partial column sums of dz (and du)
  size_t part;                 // partial products of split contractions
};

// Element counts of the padded forms: rows of a copy are padded with zeros to
// whole 16-byte pieces.
inline int64_t linear_pad(int64_t n, int dtype) {
  const int64_t m = dtype == MOE_DTYPE_F32 ? 4 : 8;
  return (n + m - 1) / m * m;
}

// Rows that are not whole 16-byte pieces at 16-byte strides: their elements are
// read one by one (and copied to padded rows for the tiles), so that their
// matrix needs the alignment of an element alone.
inline bool linear_odd_rows(int64_t width, int64_t ld, int dtype) {
  return width % linear_pad(1, dtype) || ld % linear_pad(1, dtype);
}

// Epilogue, shared by all its kernels: eight consecutive columns of one row.
struct Epilogue {
  const void *bias, *bias_up, *residual;
  void *y, *z, *z_up;
  int64_t ld_y, ld_res, ld_z;
  int N;                       // output columns
  int act;                     // moe_activation
  float limit;
  int vec;                     // every row piece of 8 columns is 16-byte aligned
};

// Arguments of the kernels for few rows and small products (linear_small.hip).
struct SmallArgs {
  const void *x, *w, *w_up;
  const void *dy, *z, *z_up;   // backward
  void *dx, *dw, *dw_up, *db, *db_up;
  int64_t M, K, ld_x, ld_dy, ld_dx;
  int64_t dx_tiles;            // set at launch
  Epilogue e;                  // backward: N, act, limit
};
constexpr int kFewRows = 16;   // rows that the few-row kernel takes

LinearSpace linear_space(const moe_linear_config &c, bool backward, bool dx, bool dw, bool db);

// Which kernels a product takes (moe_linear_product, of a checked configuration).
moe_linear_path_info linear_path(const moe_linear_config &c, int32_t product);

// Whether each launch of a call has fewer than 2^32 threads, as HIP asks (backward:
// for every gradient).
bool linear_launchable(const moe_linear_config &c, bool backward);

hipError_t launch_linear(const moe_linear_config &c, const moe_linear_weights &w, const void *x,
                         const void *residual, void *y, void *z, void *z_up, char *ws,
                         hipStream_t s);
hipError_t launch_linear_backward(const moe_linear_config &c, const moe_linear_weights &w,
                                  const void *x, const void *dy, const void *z, const void *z_up,
                                  const moe_linear_grads &g, char *ws, hipStream_t s);

// rows <= kFewRows; rows of x and w whole 16-byte pieces at 16-byte strides.
template <typename T> hipError_t launch_few_rows(const SmallArgs &a, bool dual, hipStream_t s);
// Any widths and strides.
template <typename T> hipError_t launch_small_forward(const SmallArgs &a, bool dual, hipStream_t s);
template <typename T> hipError_t launch_small_backward(SmallArgs a, bool dual, hipStream_t s);

}  // namespace moe
