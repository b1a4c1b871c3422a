// Host-side interface between the C-ABI layer (rmsnorm_api.cpp) and the RMS
// norm's kernels (rms_norm.hip). Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mscan {

constexpr int32_t kRnMaxChannels = 16384;  // 16 for each of 1024 threads

// Validated arguments of one call (see include/mamba_rmsnorm.h). A backward
// call has dy, reads h and writes dx and dresidual; an 8-bit one has scales.
struct RnCall {
  int64_t rows;
  int32_t channels, io_dtype, residual_dtype, block;
  float eps;
  const void *x, *residual, *h, *dy, *dh;
  int64_t x_row, residual_row, h_row, dy_row, dh_row;  // elements between rows
  const float* weight;
  void *y, *h_out, *dx, *dresidual;
  float *scales, *dweight;
  float* part;  // [blocks][channels] sums of dweight
  hipStream_t stream;
};
// Workspace floats of a backward call that wants dweight.
size_t rn_part_floats(int64_t rows, int32_t channels, int32_t io_dtype);
hipError_t launch_rmsnorm(const RnCall& c);

}  // namespace mscan
