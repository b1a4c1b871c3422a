// Host-side interface between the C-ABI layer (ssd_bwd_api.cpp) and the kernels
// of the SSD scan's gradients (ssd_bwd.hip). Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mscan {

// Validated arguments of one call (see include/mamba2_ssd.h).
struct SsdBwdCall {
  int32_t batch, seqlen, nheads, d_state, ngroups, io_dtype;
  const void *x, *dt, *B, *C, *dy;
  int64_t x_row, dt_row, b_row, c_row, dy_row;  // elements between rows
  const int32_t* seq_idx;  // NULL: one document per row
  const float *dt_bias, *A, *D, *state_in, *dstate_out;
  void *dx, *ddt, *dB, *dC;
  float *ddt_bias, *dA, *dD, *dstate_in;
  char* workspace;
  hipStream_t stream;
};
// Workspace bytes.
size_t ssd_bwd_ws_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t d_state, int32_t ngroups);
hipError_t launch_ssd_bwd(const SsdBwdCall& c);

}  // namespace mscan
