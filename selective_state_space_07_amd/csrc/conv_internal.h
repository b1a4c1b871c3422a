// Host-side interface between the C-ABI layer (conv_api.cpp) and the causal
// convolution's kernels (causal_conv.hip). Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mscan {

constexpr int kConvMaxParts = 4;

// Validated arguments of one call (see include/mamba_conv.h). A backward call
// has dx, and its parts are those of dy.
struct ConvCall {
  int32_t batch, seqlen, channels, taps, io_dtype, activation;
  const void* x;
  int64_t x_row;  // elements between rows
  const int32_t* seq_idx;
  const float *weight, *bias, *state_in;
  int32_t parts, part_channels[kConvMaxParts];
  void* part[kConvMaxParts];          // y, or dy
  int64_t part_row[kConvMaxParts];    // elements between their rows
  float* state_out;
  const float* dstate_out;
  void* dx;
  float *dweight, *dbias, *dstate_in;
  float* sums;  // [blocks][channels][taps] sums of dweight, then [blocks][channels] of dbias
  hipStream_t stream;
};
// Workspace floats of a backward call.
size_t conv_part_floats(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps);
hipError_t launch_conv(const ConvCall& c);
hipError_t launch_conv_step(const ConvCall& c);

}  // namespace mscan
