// Internal interface of the row norms: parameters and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ret {

constexpr int kMaxNormWidth = 16384;

struct NormParams {
  int64_t rows;
  int width, center;
  float eps, skip;
  const void *x, *y, *gate;                // y: the block's output (residual norm)
  const float *weight, *post, *scale;      // [width] or null
  void *out, *residual;                    // forward
  const void *dout, *dresidual;            // backward
  void *dx, *dy, *dgate;
  float *dweight, *dpost, *dscale;
  float* partial;  // [sums][blocks][width] column sums of the backward
};

// Column sums of a backward call: workgroups that keep one, at most.
int norm_bwd_blocks(int64_t rows, int width);

hipError_t launch_head_norm_fwd(const NormParams& p, int dtype, hipStream_t stream);
hipError_t launch_head_norm_bwd(const NormParams& p, int dtype, hipStream_t stream);
hipError_t launch_residual_norm_fwd(const NormParams& p, int dtype, hipStream_t stream);
hipError_t launch_residual_norm_bwd(const NormParams& p, int dtype, hipStream_t stream);

// out[c] = sum over rows of partial[row][c], in a fixed order
hipError_t launch_column_sum(const float* partial, int rows, int width, float* out, hipStream_t stream);

}  // namespace ret
