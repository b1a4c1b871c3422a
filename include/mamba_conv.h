/*
 * mamba_conv.h -- C ABI of the short causal convolution in libmamba_scan.so
 * (MI355X, gfx950): the depthwise convolution over time that stands in front
 * of a scan, on its own, for the channels x, B and C of a Mamba-2 block, with
 * its gradients and its one-token form. (mamba_scan_fwd has the Mamba-1
 * block's inside.) Status codes, threading, stream and error conventions are
 * those of mamba_scan.h (validation before any HIP call, MAMBA_ERR_* codes,
 * the thread's detail in mamba_scan_last_error(), no fallback of any kind).
 *
 * The operation, per batch row and channel c, with x before the first token
 * taken from state_in (zeros where that is NULL):
 *
 *   u_t = bias[c] + sum over j < taps of weight[c][j] x_(t - taps + 1 + j)
 *   y_t = silu(u_t) (MAMBA_ACT_SILU) or u_t (MAMBA_ACT_NONE)
 *
 * silu and its derivative are 0 at the lowest values, and at -inf as well. With
 * seq_idx (packed documents) a new document starts wherever an id differs from
 * the one before it: what stands before it is zero for its tokens, whatever it
 * was. The state is the last taps - 1 inputs, oldest first, exact, and 0 for
 * those that are not of the last document.
 *
 * Sums are float32; outputs are rounded to the io type once. Results are bitwise
 * reproducible run to run.
 *
 * Layouts and limits:
 *   x                [batch][seqlen][channels] io, rows x_stride elements apart
 *                    (at least channels, at most 2^24), so that it can be
 *                    columns of a wider tensor
 *   parts            1 to MAMBA_CONV_MAX_PARTS tensors that the channels of y
 *                    (or dy) are split over, in order: part_channels[i] of them
 *                    in part i, which add up to channels
 *   y                one pointer for each part: [batch][seqlen][part_channels[i]]
 *                    io, contiguous
 *   weight           [channels][taps] float32, taps 2, 3 or 4
 *   bias             [channels] float32, or NULL (zeros)
 *   seq_idx          [batch][seqlen] int32, or NULL (one document per row)
 *   states           [batch][channels][taps - 1] float32
 * Element alignment is enough (pointers, rows and parts at multiples of four
 * elements run faster). channels <= 2^20; batch <= 2^24; batch * seqlen < 2^30. Inputs
 * may overlap one another, outputs nothing.
 */
#ifndef MAMBA_CONV_H
#define MAMBA_CONV_H

#include <stddef.h>
#include <stdint.h>

#include "mamba_gnorm.h" /* enum mamba_activation */
#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_CONV_MAX_PARTS 4

/* state_in may be NULL (zeros), state_out too (not written). */
int mamba_conv_fwd(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype,
                   int32_t activation, const void* x, int64_t x_stride, const int32_t* seq_idx, const float* weight,
                   const float* bias, const float* state_in, int32_t parts, const int32_t* part_channels,
                   void* const* y, float* state_out, void* stream);

/* Bytes of device workspace mamba_conv_bwd needs (0 for arguments it rejects):
   one partial sum of dweight and dbias per workgroup. */
size_t mamba_conv_bwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype);

/*
 * Gradients of mamba_conv_fwd with the same arguments; nothing of the forward
 * call is kept.
 *   dy               one pointer for each part, rows dy_stride[i] elements apart
 *   dstate_out       gradient of the forward's state_out, or NULL (zeros)
 *   dx               [batch][seqlen][channels] io, contiguous
 *   dweight          [channels][taps] float32
 *   dbias            [channels] float32, or NULL (not wanted)
 *   dstate_in        gradient of state_in, or NULL (not wanted)
 *   workspace        >= mamba_conv_bwd_workspace_bytes(...) bytes, 256-byte aligned
 */
int mamba_conv_bwd(int32_t batch, int32_t seqlen, int32_t channels, int32_t taps, int32_t io_dtype,
                   int32_t activation, const void* x, int64_t x_stride, const int32_t* seq_idx, const float* weight,
                   const float* bias, const float* state_in, int32_t parts, const int32_t* part_channels,
                   const void* const* dy, const int64_t* dy_stride, const float* dstate_out, void* dx, float* dweight,
                   float* dbias, float* dstate_in, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token per batch row: x [batch][channels] with rows x_stride apart, y one
 * [batch][part_channels[i]] for each part. state_in is required; state_out may
 * be exactly state_in (in place).
 */
int mamba_conv_step(int32_t batch, int32_t channels, int32_t taps, int32_t io_dtype, int32_t activation, const void* x,
                    int64_t x_stride, const float* weight, const float* bias, const float* state_in, int32_t parts,
                    const int32_t* part_channels, void* const* y, float* state_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_CONV_H */
