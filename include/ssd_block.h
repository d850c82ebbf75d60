/*
 * ssd_block.h -- C ABI of the operators a Mamba-2 block needs around the scan
 * to be trained and served (GB300, sm_103a): the residual RMSNorm before the
 * block, the gated grouped RMSNorm after its scan, the causal conv1d's
 * backward and one-token step, the projections and gradient clipping.
 *
 * Conventions are those of ssd_scan.h (same library, same error codes and
 * ssd_last_error(), dtype arguments, streams): device pointers owned by the
 * caller, nothing kept after the call returns, everything enqueued on
 * `stream`, arguments validated before anything is launched, no host
 * synchronisation.  Differences are stated at each call.  "x dtype" is the
 * dtype argument (fp32 or bf16).  Every sum, statistic and gradient of a
 * parameter is accumulated in fp32 or more; each output is rounded once.
 * No call uses atomics on values: equal inputs give equal bits.
 * Workspace: device memory of at least the queried bytes, 256-byte aligned,
 * used only by the call's own work on `stream`.
 */
#ifndef SSD_BLOCK_H
#define SSD_BLOCK_H

#include "ssd_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this header's calls (ssd_abi_version() is that of ssd_scan.h). */
#define SSD_BLOCK_ABI_VERSION 1
int ssd_block_abi_version(void);

/* ---------------------------------------------------------------------------
 * Residual RMSNorm before a block (pre-norm with its residual stream):
 *   r = residual + scale * x         (scale per channel, or 1)
 *   y = weight * r / sqrt(mean_c r^2 + eps)
 * r is stored in the residual's type and the norm is that of the stored
 * value, so that the backward, which reads r, differentiates exactly the
 * function that ran.
 *   x             [rows, dim] x dtype
 *   residual      [rows, dim] residual_dtype, or NULL (= 0)
 *   scale         [dim] float, or NULL (= 1)
 *   weight        [dim] float
 *   y             [rows, dim] x dtype (written)
 *   residual_out  [rows, dim] residual_dtype (written; may be residual)
 * residual_dtype is fp32 or the x dtype.  rows in [1, 2^31), dim in
 * [1, 16384], any value; 16-byte aligned rows (dim a multiple of 8) take wide
 * accesses, others one element at a time.  Pointers aligned to their element.
 * ------------------------------------------------------------------------- */
int ssd_add_rmsnorm_fwd(const void *x, const void *residual, const float *scale,
                        const float *weight, float eps, int64_t rows, int dim,
                        ssd_dtype_t dtype, ssd_dtype_t residual_dtype, void *y,
                        void *residual_out, void *stream);

/* Its backward.  With n = r / sqrt(mean r^2 + eps), g = weight * dy:
 *   dresidual = dresidual_out + (g - n * mean_c(g n)) / sqrt(mean r^2 + eps)
 *   dx = scale * dresidual,  dweight = sum_rows dy * n,
 *   dscale = sum_rows dresidual * x
 *   dy             [rows, dim] x dtype: gradient of y
 *   dresidual_out  [rows, dim] residual_dtype: gradient of residual_out, or
 *                  NULL (= 0)
 *   residual_out   the forward's, x the forward's x (required iff dscale)
 *   dx             [rows, dim] x dtype, dresidual [rows, dim] residual_dtype
 *                  (each may be NULL; dresidual may be dresidual_out)
 *   dweight        [dim] float; dscale [dim] float (required iff scale)
 * All written, not accumulated. */
size_t ssd_add_rmsnorm_bwd_workspace_bytes(int64_t rows, int dim);
int ssd_add_rmsnorm_bwd(const void *dy, const void *dresidual_out,
                        const void *residual_out, const void *x,
                        const float *scale, const float *weight, float eps,
                        int64_t rows, int dim, ssd_dtype_t dtype,
                        ssd_dtype_t residual_dtype, void *dx, void *dresidual,
                        float *dweight, float *dscale, void *workspace,
                        size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Gated RMSNorm after the scan, over groups of group_size channels:
 *   norm_before_gate = 0:  u = y * silu(z);  out = weight * u / rms(u)
 *   norm_before_gate = 1:  out = weight * y / rms(y) * silu(z)
 *   rms(u) = sqrt(mean over the channel's group of u^2 + eps)
 * (the two orders of norm_before_gate in the block call of state-spaces/mamba
 * issue #647; the first, applied to an ungated scan output, is that block's
 * norm).  z NULL: no gate.
 *   y, z    [batch, seqlen, dim] x dtype, the channels of a token dense, with
 *           element strides between tokens and batch rows (z is typically a
 *           slice of the input projection); strides >= 0
 *   weight  [dim] float
 *   out     [batch, seqlen, dim] x dtype, dense (written; may be y if dense)
 * group_size in [1, 16384] divides dim; batch * seqlen in [1, 2^31), dim /
 * group_size <= 65535. */
int ssd_gated_rmsnorm_fwd(const void *y, ssd_stride_t y_stride, const void *z,
                          ssd_stride_t z_stride, const float *weight, float eps,
                          int64_t batch, int64_t seqlen, int dim, int group_size,
                          int norm_before_gate, ssd_dtype_t dtype, void *out,
                          void *stream);

/* Its backward for the upstream gradient dout ([batch, seqlen, dim] x dtype,
 * dense): dy (dense), dz (strided: it can be written into a slice of the
 * projection's gradient; required iff z), both x dtype, and dweight [dim]
 * float.  All written, not accumulated. */
size_t ssd_gated_rmsnorm_bwd_workspace_bytes(int64_t batch, int64_t seqlen,
                                             int dim, int group_size);
int ssd_gated_rmsnorm_bwd(const void *dout, const void *y, ssd_stride_t y_stride,
                          const void *z, ssd_stride_t z_stride,
                          const float *weight, float eps, int64_t batch,
                          int64_t seqlen, int dim, int group_size,
                          int norm_before_gate, ssd_dtype_t dtype, void *dy,
                          void *dz, ssd_stride_t dz_stride, float *dweight,
                          void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_BLOCK_H */
