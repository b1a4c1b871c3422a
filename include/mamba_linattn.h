/*
 * mamba_linattn.h -- C ABI of linear attention with a decay for each head in
 * libmamba_scan.so (MI355X, gfx950): a whole sequence, its gradients, and one
 * token. Status codes, threading, stream and error conventions are those of
 * mamba_scan.h (validation before any HIP call, MAMBA_ERR_* codes, the
 * thread's detail in mamba_scan_last_error(), no fallback of any kind).
 *
 * The operation, per batch row b and head h with q/k head
 * g = h / (nheads / ngroups), lam = exp(log_decay[h]) and a state matrix
 * S[d_v][d_k]:
 *
 *   S        = lam * S + v[b,t,h,:] (outer) k[b,t,g,:]
 *   y[b,t,h] = scale * S q[b,t,g,:]
 *
 * It is the recurrence of mamba2_ssd.h with a decay that depends on the head
 * alone, for any head sizes, with gradients. log_decay is meant to be <= 0
 * (-inf: no memory). Values above 0 grow the state and are not refused; from
 * 1.38 on lam^64 is beyond float32, and NaN may come out where the state itself
 * would not be. The decays are constants of an architecture here: no gradient
 * is defined for them.
 *
 * A sequence is evaluated in chunks of 64 tokens on the matrix cores with
 * float32 accumulation. For bfloat16 io the operands of y's two products that
 * are not inputs (the decayed scores q.k, and S) are two bfloat16 parts each, 16
 * bits, so that outputs have the error of their own rounding; the state itself
 * is summed in float32 (w v enters its products as three parts). For float32 io
 * each operand is three bfloat16 parts, to float32 accuracy; what lies below
 * 1e-38 in a value is lost there. The result equals the recurrence up to
 * rounding, is bitwise reproducible and does not depend on which outputs are
 * wanted. An infinity may come out as NaN in the outputs and states that it
 * enters (a part of what it meets may be 0); with bfloat16 io one in v or in a
 * state stays one. A token's output depends only on the tokens of its own document
 * up to it: where others hold infinities or NaN it has the bits that it has
 * without them, and so have the gradients.
 *
 * Layouts and limits of all calls:
 *   q, k         [batch][seqlen][ngroups][d_k] io, 16-byte aligned
 *   v, y         [batch][seqlen][nheads][d_v]  io, 16-byte aligned
 *   log_decay    [nheads] float32
 *   state        [batch][nheads][d_v][d_k] float32, 16-byte aligned
 *   seq_idx      [batch][seqlen] int32, or NULL
 * The rows (b, t) of q, k, v and dy are *_stride elements apart (at least
 * their own width, at most 2^24, a multiple of 16 bytes), so that they can be
 * columns of one projection's output; the other tensors are contiguous.
 * d_k and d_v are multiples of 8 up to 128; ngroups divides nheads;
 * nheads <= 4096, batch * nheads <= 2^20, seqlen <= 2^30, batch * seqlen < 2^31.
 * The inputs may overlap one another, the outputs nothing.
 */
#ifndef MAMBA_LINATTN_H
#define MAMBA_LINATTN_H

#include <stddef.h>
#include <stdint.h>

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace mamba_linattn_fwd needs: the states between the
   segments a long sequence of few heads is split into (0 where it is not
   split, and for arguments the call rejects). */
size_t mamba_linattn_fwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups,
                                         int32_t d_k, int32_t d_v, int32_t io_dtype);

/*
 * Whole sequence.
 *   seq_idx      document ids, or NULL: the state restarts from zero before
 *                every token whose id differs from the previous token's (packed
 *                documents, as mamba2_ssd_fwd_seq)
 *   state_in     the state before the first token, or NULL (zeros)
 *   state_out    the state after the last token, or NULL (not written); may be
 *                exactly state_in
 *   workspace    >= mamba_linattn_fwd_workspace_bytes(...) bytes, 256-byte
 *                aligned (NULL where that is 0)
 */
int mamba_linattn_fwd(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v,
                      int32_t io_dtype, float scale, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, const int32_t* seq_idx,
                      const float* log_decay, const float* state_in, void* y, float* state_out, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Bytes of device workspace mamba_linattn_bwd needs: segment states as above,
   and float32 dq and dk of every head where heads share them. */
size_t mamba_linattn_bwd_workspace_bytes(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups,
                                         int32_t d_k, int32_t d_v, int32_t io_dtype);

/*
 * Gradients of mamba_linattn_fwd with the same arguments; nothing of the
 * forward call is kept.
 *   dy           like v: the gradient of y
 *   dstate_out   the gradient of the final state, like state, or NULL (zeros)
 *   dq, dk       [batch][seqlen][ngroups][d_k] io, summed over a group's heads
 *   dv           [batch][seqlen][nheads][d_v] io
 *   dstate_in    the gradient of state_in, like state, or NULL (not written)
 */
int mamba_linattn_bwd(int32_t batch, int32_t seqlen, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v,
                      int32_t io_dtype, float scale, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, const int32_t* seq_idx,
                      const float* log_decay, const float* state_in, const void* dy, int64_t dy_stride,
                      const float* dstate_out, void* dq, void* dk, void* dv, float* dstate_in, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * One token per batch row: the recurrence itself, for seqlen 1. state_in and
 * state_out are required; state_out may be exactly state_in (in place). The
 * batch rows of q, k and v are *_stride elements apart (any multiple of the
 * element size; io pointers need their element's alignment only). No workspace.
 * batch * nheads * d_v < 2^31.
 */
int mamba_linattn_step(int32_t batch, int32_t nheads, int32_t ngroups, int32_t d_k, int32_t d_v, int32_t io_dtype,
                       float scale, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const float* log_decay, const float* state_in, void* y, float* state_out,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_LINATTN_H */
