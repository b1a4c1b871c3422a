// Host-side interface between the C-ABI layer (gnorm_api.cpp) and the group
// norm kernels (group_norm.hip). Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mscan {

constexpr int32_t kGnMaxGroup = 16384;  // channels of one group: 16 for each of 1024 threads

// Validated arguments of one call (see include/mamba_gnorm.h). A backward call
// has dy and writes out (dx), dz and, through part, dweight and dbias.
struct GnCall {
  int64_t rows;
  int32_t channels, groups, io_dtype, activation, gate, center;
  float eps;
  const void *x, *z, *dy;
  int64_t x_row, z_row, dy_row;  // elements between rows
  const float *weight, *bias;
  void *out, *dz;
  float *dweight, *dbias;  // NULL: not wanted
  float* part;             // [blocks][channels] sums of dweight, then of dbias
  hipStream_t stream;
};
// Workspace floats of a backward call that wants `sums` (0, 1 or 2) of dweight and dbias.
size_t gn_part_floats(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int sums);
hipError_t launch_gnorm(const GnCall& c);

}  // namespace mscan
