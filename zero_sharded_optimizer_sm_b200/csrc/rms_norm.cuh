// The root-mean-square norm of a layer's input with the residual stream's
// addition, forward and backward: launch arguments and launchers.
//
//   h = x + residual (rounded to its type; x where there is no residual)
//   rstd = (mean(h^2) + eps)^(-1/2),  y = h rstd w
//   xh = h rstd,  g = dy w
//   dx = rstd (g - xh mean(g xh)) + dh,  dw = sum over the rows of dy xh
#pragma once

#include "mx8.cuh"

namespace zsm {

struct RmsNormArgs {
  const void *x, *residual;  // of `type`; residual may be null
  int type;
  int64_t rows, cols, ld_x, ld_residual;
  const void* weight;
  int w_type;
  bool w_aligned;  // to 16 bytes
  float eps;
  void *y, *h;  // of `type`; any of the five results may be null (or have null codes)
  int64_t ld_y, ld_h;
  Mx8Matrix y8, h8;
  float* rstd;
};

struct RmsNormBackwardArgs {
  const void *dy, *h, *dh;  // of `type`; h null: h8; dh may be null
  int type;
  int64_t rows, cols, ld_dy, ld_h, ld_dh;
  uintptr_t dy_end, h_end, dh_end;  // behind the matrices' last elements
  Mx8Matrix h8;
  const void* weight;
  int w_type;
  bool w_aligned;  // to 16 bytes
  const float* rstd;
  void *dx, *dw;
  int64_t ld_dx;
  int dw_type;
  void* workspace;
};

cudaError_t launch_rms_norm(const RmsNormArgs& a, int sm_count, cudaStream_t s);
cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, int sm_count, cudaStream_t s);
// Bytes of workspace of the backward pass, on any device.
int64_t rms_norm_backward_workspace(int64_t rows, int64_t cols);

}  // namespace zsm
