// Host-side interface between the C-ABI layer (linattn_api.cpp) and the
// linear-attention kernels (lin_attn.hip). Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mscan {

// An io operand [batch][seqlen][heads or groups][dim]: consecutive tokens are
// `row` elements apart, batch rows seqlen * row.
struct LaOperand {
  const void* p;
  int64_t row;
  bool per_group;  // one head for each group of heads (else one for each head)
};

// One mixing sum out_t = sum_s w(t, s) (q_t . k_s) v_s with its carried state
// S[vd][kd] = sum_s w'(s) v_s k_s^T, forwards or backwards in time. The
// forward call is one of these, the backward three (lin_attn.hip).
struct LaRole {
  LaOperand q, k, v;
  int32_t kd, vd;          // elements of q and k, of v and out
  void* out;               // [batch][seqlen][nheads][vd]: io, or float32 where out_f32
  bool out_f32;
  const float* state_in;   // [batch][nheads][vd][kd] ([kd][vd] where state_t), or NULL (zeros)
  bool state_t;
  float* state_out;        // [batch][nheads][vd][kd], or NULL
  float sc_out, sc_kv;     // factors on what is read out, and on what enters the state
  bool rev;                // from the last token to the first
  int32_t off;             // 1: the incoming state stands one step before the first token; 0: at it
  bool keeps;              // a role whose state may be returned, whether this call wants it or not
};

struct LaCall {
  int32_t batch, seqlen, nheads, ngroups, io_dtype;
  const int32_t* seq_idx;  // NULL: one document per row
  const float* log_decay;
  int32_t nroles;
  LaRole role[3];
  float* workspace;
  hipStream_t stream;
};

// The sequence split: segments of seg_chunks chunks of 64 tokens, run side by
// side; with more than one, a first pass sums each segment's state.
struct LaPlan {
  int32_t nseg, seg_chunks;
};
LaPlan la_plan(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v, int32_t nroles);
// Workspace floats of the segment states and flags (0 for one segment).
size_t la_ws_floats(const LaPlan& p, int32_t batch, int32_t nheads, int32_t d_k, int32_t d_v, int32_t nroles);
hipError_t launch_la(const LaCall& c, const LaPlan& p);

// out[row][g][d] = sum over the heads of group g of part[row][h][d] (float32),
// for the gradients of shared q and k heads.
hipError_t launch_la_head_sum(int64_t rows, int32_t nheads, int32_t ngroups, int32_t d, int32_t io_dtype,
                              const float* part, void* out, hipStream_t stream);

struct LaStepCall {
  int32_t batch, nheads, ngroups, d_k, d_v, io_dtype;
  float scale;
  const void *q, *k, *v;
  int64_t q_row, k_row, v_row;  // elements between batch rows
  const float *log_decay, *state_in;
  void* y;
  float* state_out;
  hipStream_t stream;
};
hipError_t launch_la_step(const LaStepCall& c);

}  // namespace mscan
