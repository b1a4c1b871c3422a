/*
 * mamba_gnorm.h -- C ABI of the group norm with an activation and a gate in
 * libmamba_scan.so (MI355X, gfx950): the norm behind a scan (gated, per head
 * or over all channels) and its gradients. Status codes, threading, stream and
 * error conventions are those of mamba_scan.h (validation before any HIP call,
 * MAMBA_ERR_* codes, the thread's detail in mamba_scan_last_error(), no
 * fallback of any kind).
 *
 * The operation, per row (token) and group of channels / groups neighbouring
 * channels, with act the activation and a = act(z):
 *
 *   u = x a (MAMBA_GATE_FIRST) or x
 *   m = mean of u over the group (0 where center is 0)
 *   n = (u - m) / sqrt(mean of (u - m)^2 + eps) * weight + bias
 *   y = n a (MAMBA_GATE_AFTER), n (MAMBA_GATE_FIRST) or act(n) (MAMBA_GATE_NONE)
 *
 * silu and its derivative are 0 at the lowest values, and at -inf as well, so
 * that either closes a gate. Each row is a sample of its own: a token's output
 * depends on that token alone. One group and center 0 is an RMS norm; with
 * MAMBA_GATE_FIRST and silu it is the norm of a Mamba-2 block behind
 * mamba2_ssd_fwd.
 *
 * Statistics, sums and gradients of the parameters are float32 throughout
 * (the mean first, then the squares of the differences; values whose squares
 * leave float32 are taken times a power of two); outputs are rounded to the io
 * type once. Results are bitwise reproducible run to run.
 *
 * Layouts and limits:
 *   x, z, dy         [rows][channels] io, rows *_stride elements apart (at least
 *                    channels, at most 2^24), so that they can be columns of
 *                    one wider tensor; element alignment is enough (16-byte
 *                    alignment of pointers and rows and groups of a multiple of
 *                    16 bytes run faster)
 *   y, dx, dz        [rows][channels] io, contiguous
 *   weight, bias     [channels] float32, or NULL (1 and 0)
 * groups divides channels; a group has at most 16384 channels; channels <=
 * 2^20; eps >= 0; rows * groups < 2^31. Inputs may overlap one another, outputs nothing.
 */
#ifndef MAMBA_GNORM_H
#define MAMBA_GNORM_H

#include <stddef.h>
#include <stdint.h>

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

enum mamba_activation { MAMBA_ACT_NONE = 0, MAMBA_ACT_SILU = 1, MAMBA_ACT_SIGMOID = 2 };
enum mamba_gate { MAMBA_GATE_NONE = 0, MAMBA_GATE_AFTER = 1, MAMBA_GATE_FIRST = 2 };

/* z is NULL exactly where gate is MAMBA_GATE_NONE. */
int mamba_gnorm_fwd(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int32_t activation,
                    int32_t gate, int32_t center, float eps, const void* x, int64_t x_stride, const void* z,
                    int64_t z_stride, const float* weight, const float* bias, void* y, void* stream);

/* Bytes of device workspace mamba_gnorm_bwd needs: one partial sum of each of
   dweight and dbias that is wanted per workgroup (0 where neither is, and for
   arguments the call rejects). */
size_t mamba_gnorm_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype,
                                       int32_t want_dweight, int32_t want_dbias);

/*
 * Gradients of mamba_gnorm_fwd with the same arguments; nothing of the forward
 * call is kept.
 *   dx               gradient of x
 *   dz               gradient of z; NULL exactly where gate is MAMBA_GATE_NONE
 *   dweight, dbias   [channels] float32, or NULL (not wanted; also where weight
 *                    or bias is NULL they may be asked for)
 *   workspace        >= mamba_gnorm_bwd_workspace_bytes(...) bytes, 256-byte
 *                    aligned (NULL where that is 0)
 */
int mamba_gnorm_bwd(int64_t rows, int32_t channels, int32_t groups, int32_t io_dtype, int32_t activation,
                    int32_t gate, int32_t center, float eps, const void* x, int64_t x_stride, const void* z,
                    int64_t z_stride, const float* weight, const float* bias, const void* dy, int64_t dy_stride,
                    void* dx, void* dz, float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_GNORM_H */
