/*
 * ssd_delta.h -- C ABI of the gated delta rule (GB300, sm_103a): the chunked
 * scan, its backward and its one-token step, next to ssd_scan.h's SSD scan.
 * One independent recurrence per batch row b and head h, queries and keys
 * shared by groups of heads (group h / (nheads / ngroups)):
 *
 *   S' = exp(g_t) S_{t-1}                        S [headdim, dstate]
 *   u_t = beta_t (v_t - S' k_t)                  what v_t adds to the state's answer
 *   S_t = S' + u_t (outer) k_t
 *   out_t = scale * S_t q_t
 *
 * Conventions are those of ssd_scan.h (same library, error codes and
 * ssd_last_error(), dtype arguments, streams): device pointers owned by the
 * caller, nothing kept after the call returns, everything enqueued on `stream`,
 * arguments validated before anything is launched, no host synchronisation, no
 * atomics on values (equal inputs give equal bits).  "x dtype" is the dtype
 * argument, fp32 or bf16; every sum, the states and the decays are held in
 * fp32 or more, and each output is rounded once.  The tensor cores' factors that are
 * computed (the state, the corrections u, the chunks' matrices, their gradients)
 * enter the products as sums of bf16 terms: three for fp32 tensors, whose results are
 * off by 1e-7 to 6e-7 of their norm as fp32 arithmetic is; two for bf16 ones, 2^-18
 * of a factor, and so is what the workspace keeps for the backward.  With bf16
 * tensors the fp32 results (final_states, dg, dbeta, d_initial_states) are therefore
 * off by 2e-6 to 6e-6 of their norm: far less than the tensors' own rounding, but not
 * an fp32 computation's, which the same values as fp32 tensors give.
 * Pointers are aligned to their element (dq and dk to two; rows on 16 bytes take wide
 * accesses), the workspace to 256 bytes.  An output (and the workspace) may share no memory with an input or
 * another output, but final_states may be initial_states, d_initial_states may be
 * dfinal_states, and the step's out its v: others are refused (SSD_ERR_ARG).
 *
 * Tensors:
 *   q, k          [batch, seqlen, ngroups, dstate] x dtype
 *   v             [batch, seqlen, nheads, headdim] x dtype
 *                 each token's part dense, element strides between batch rows
 *                 and tokens (>= 0), e.g. slices of a projection
 *   g, beta       [batch, seqlen, nheads] float, dense.  g is the logarithm of
 *                 the decay: at most 0 in use, larger values grow the state; below
 *                 -104 (exp is 0 in fp32) the state starts anew, and g has no
 *                 gradient there
 *   seq_idx       [batch, seqlen] int32 or NULL: the state is set to zero before
 *                 token t whenever seq_idx[b,t] != seq_idx[b,t-1] (times a decay of
 *                 0: a state that is not finite stays so)
 *   initial_states, final_states  [batch, nheads, headdim, dstate] float
 * Sizes: dstate in [1, 128], headdim in [1, 2048], nheads a multiple of ngroups,
 * batch * nheads * chunks < 2^31 (chunks of 64 tokens for bf16, 32 for fp32).
 * Keys of unit length (and beta in [0, 2]) keep the recurrence stable; the call
 * does not normalise them.  An infinity or NaN spreads, as in any chunked form,
 * to its chunk's other tokens of its head, and to those after it, past starts of
 * documents too (its products with zeros are NaN).  Finite values do not count as such
 * up to the end of the fp32 range, but for a bf16 dv that rounds to an infinity: the
 * other gradients of its chunk are then not finite.
 */
#ifndef SSD_DELTA_H
#define SSD_DELTA_H

#include "ssd_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_DELTA_ABI_VERSION 1
int ssd_delta_abi_version(void);

/* The scan.  out [batch, seqlen, nheads, headdim] x dtype, dense (written);
 * final_states written, or NULL.
 * keep: nonzero if the workspace is to hold what ssd_delta_scan_bwd would
 * otherwise compute again (each chunk's triangular inverse and scores, first
 * state and corrections): it is then passed there as `saved`, unchanged.
 * aligned (workspace queries): nonzero if q, k and v (and for the backward dout)
 * have every token's rows on 16 bytes (pointer, strides and row lengths) and no
 * stride of 0 along a length above 1; others may be copied in the workspace.
 * workspace_bytes: 0 on bad sizes. */
size_t ssd_delta_scan_workspace_bytes(int64_t batch, int64_t seqlen, int nheads,
                                      int headdim, int dstate, int ngroups,
                                      ssd_dtype_t dtype, int keep, int aligned);
int ssd_delta_scan_fwd(const void *q, ssd_stride_t q_stride, const void *k,
                       ssd_stride_t k_stride, const void *v,
                       ssd_stride_t v_stride, const float *g, const float *beta,
                       float scale, const float *initial_states,
                       const int32_t *seq_idx, int64_t batch, int64_t seqlen,
                       int nheads, int headdim, int dstate, int ngroups,
                       ssd_dtype_t dtype, void *out, float *final_states,
                       int keep, void *workspace, size_t workspace_bytes,
                       void *stream);

/* Its backward for the upstream gradients dout of out ([batch, seqlen, nheads,
 * headdim] x dtype, dense) and dfinal_states of final_states (or NULL: zero);
 * the forward's other arguments as they were.
 *   saved  the workspace of a forward with keep on the same inputs (read), or
 *          NULL: the forward is computed again
 *   dq, dk [batch, seqlen, ngroups, dstate], dv [batch, seqlen, nheads, headdim]
 *          x dtype; dg, dbeta [batch, seqlen, nheads] float: all dense
 *   d_initial_states  [batch, nheads, headdim, dstate] float, or NULL
 * All written, not accumulated. */
size_t ssd_delta_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen,
                                          int nheads, int headdim, int dstate,
                                          int ngroups, ssd_dtype_t dtype,
                                          int saved, int aligned);
int ssd_delta_scan_bwd(const void *dout, const float *dfinal_states,
                       const void *q, ssd_stride_t q_stride, const void *k,
                       ssd_stride_t k_stride, const void *v,
                       ssd_stride_t v_stride, const float *g, const float *beta,
                       float scale, const float *initial_states,
                       const int32_t *seq_idx, int64_t batch, int64_t seqlen,
                       int nheads, int headdim, int dstate, int ngroups,
                       ssd_dtype_t dtype, const void *saved, size_t saved_bytes,
                       void *dq, void *dk, void *dv, float *dg, float *dbeta,
                       float *d_initial_states, void *workspace,
                       size_t workspace_bytes, void *stream);

/* One token per batch row, from a prompt's final states: q, k [batch, ngroups,
 * dstate], v, out [batch, nheads, headdim] x dtype, g, beta [batch, nheads]
 * float, dense; state [batch, nheads, headdim, dstate] float, moved on in
 * place.  Tokens are computed as the recurrence is written: infinities and NaN
 * stay in the rows of the state that they reach. */
int ssd_delta_decode_step(const void *q, const void *k, const void *v,
                          const float *g, const float *beta, float scale,
                          float *state, int64_t batch, int nheads, int headdim,
                          int dstate, int ngroups, ssd_dtype_t dtype, void *out,
                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_DELTA_H */
