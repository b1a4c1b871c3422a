/*
 * mamba_rmsnorm.h -- C ABI of the RMS norm with the residual's addition in
 * libmamba_scan.so (MI355X, gfx950): what stands between two blocks, with its
 * gradients and with an output in 8 bits for a quantised projection. Status
 * codes, threading, stream and error conventions are those of mamba_scan.h
 * (validation before any HIP call, MAMBA_ERR_* codes, the thread's detail in
 * mamba_scan_last_error(), no fallback of any kind).
 *
 * The operation, per row (token):
 *
 *   h = x + residual               (h = x where residual is NULL)
 *   y = h / sqrt(mean of h^2 + eps) * weight
 *
 * y is taken of the float32 sum, before h is rounded to its type. Sums are
 * float32 throughout (rows whose squares leave float32 are taken times a power
 * of two); outputs are rounded once. Results are bitwise reproducible run to run.
 *
 * Layouts and limits:
 *   x, dy            [rows][channels] io, rows *_stride elements apart (at least
 *                    channels, at most 2^24), so that they can be columns of one
 *                    wider tensor
 *   residual         likewise, of type residual_dtype: MAMBA_F32, or MAMBA_BF16
 *                    where io_dtype is MAMBA_BF16
 *   h, dh            of residual_dtype; as inputs with strides, as outputs contiguous
 *   y, dx            [rows][channels] io, contiguous
 *   weight           [channels] float32, or NULL (ones)
 * channels <= 16384; rows < 2^31; eps >= 0. Element alignment is enough
 * (16-byte alignment of pointers and rows runs faster), but for
 * mamba_rmsnorm_fp8. Inputs may overlap one another; outputs nothing, except
 * that h (dresidual) may be exactly residual (dh) with the same rows.
 */
#ifndef MAMBA_RMSNORM_H
#define MAMBA_RMSNORM_H

#include <stddef.h>
#include <stdint.h>

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* h may be NULL (not written). */
int mamba_rmsnorm_fwd(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                      const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                      const float* weight, void* y, void* h, void* stream);

/*
 * The same with y in 8 bits: y8 [rows][channels] as OCP e4m3 (no infinities, up
 * to 448) times a scale, one for each row (block 0) or for each 128 neighbouring
 * channels of a row (block 128; the last block may be shorter):
 *   scales           [rows][1] or [rows][ceil(channels / 128)] float32: the
 *                    block's largest |y| / 448, at least 2^-126; 1 where all are 0;
 *                    NaN where one is
 * channels must be a multiple of 16; pointers and rows 16-byte aligned.
 */
int mamba_rmsnorm_fp8(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                      int32_t block, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                      const float* weight, void* y8, float* scales, void* h, void* stream);

/* Bytes of device workspace mamba_rmsnorm_bwd needs: one partial sum of dweight
   per workgroup where it is wanted (0 where it is not, and for arguments the
   call rejects). */
size_t mamba_rmsnorm_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype,
                                         int32_t want_dweight);

/*
 * Gradients of mamba_rmsnorm_fwd from the h that it returned.
 *   h                [rows][channels] of residual_dtype
 *   dy               gradient of y, io
 *   dh               gradient that reaches h from behind, or NULL (zeros)
 *   dresidual        gradient of residual, of residual_dtype: dh and the norm's
 *   dx               the same as io; NULL: not wanted (where the types agree
 *                    dresidual is it). At least one of the two
 *   dweight          [channels] float32, or NULL (not wanted)
 *   workspace        >= mamba_rmsnorm_bwd_workspace_bytes(...) bytes, 256-byte
 *                    aligned (NULL where that is 0)
 */
int mamba_rmsnorm_bwd(int64_t rows, int32_t channels, int32_t io_dtype, int32_t residual_dtype, float eps,
                      const void* h, int64_t h_stride, const float* weight, const void* dy, int64_t dy_stride,
                      const void* dh, int64_t dh_stride, void* dx, void* dresidual, float* dweight, void* workspace,
                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_RMSNORM_H */
