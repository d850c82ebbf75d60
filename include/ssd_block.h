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
 *   y             [rows, dim] x dtype (written; no other tensor's memory)
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

/* ---------------------------------------------------------------------------
 * Backward of ssd_causal_conv1d (ssd_scan.h) for the upstream gradient dout of
 * its out, the forward's other arguments as they were.  With pre = the
 * forward's value before act, recomputed, and dpre = dout * act'(pre):
 *   dx[b,s,c]    = sum_k weight[c,k] dpre[b, s+width-1-k, c]
 *   dweight[c,k] = sum_{b,t} dpre[b,t,c] x[b, t-width+1+k, c]
 *   dbias[c]     = sum_{b,t} dpre[b,t,c]
 * over the taps that the forward counts (inside the sequence and, with
 * seq_idx, in token t's document).
 *   dout, x, dx  [batch, seqlen, channels] x dtype, channels dense, with
 *                strides as for the forward's x (multiples of 16 bytes); dx may
 *                be a slice of the projection's gradient, and must not overlap
 *                x or dout
 *   dweight      [channels, width] float;  dbias [channels] float or NULL
 * All written, not accumulated.  channels a multiple of 8, width 1..8; dout,
 * x and dx 16-byte aligned. */
size_t ssd_causal_conv1d_bwd_workspace_bytes(int64_t batch, int64_t seqlen,
                                             int channels, int width);
int ssd_causal_conv1d_bwd(const void *dout, ssd_stride_t dout_stride,
                          const void *x, ssd_stride_t x_stride,
                          const float *weight, const float *bias,
                          const int32_t *seq_idx, int64_t batch, int64_t seqlen,
                          int channels, int width, int silu, ssd_dtype_t dtype,
                          void *dx, ssd_stride_t dx_stride, float *dweight,
                          float *dbias, void *workspace, size_t workspace_bytes,
                          void *stream);

/* One token of the conv per batch row, next to ssd_decode_step:
 *   out[b,c] = act(bias[c] + sum_{k<width-1} weight[c,k] conv_state[b,k,c]
 *                  + weight[c,width-1] x[b,c])
 * and conv_state, the last width-1 inputs of the sequence, oldest first,
 * moves on by one (in place).  After a prompt it is the prompt's last width-1
 * inputs (zeros before its start).
 *   x           [batch, channels] x dtype, rows x_row_stride elements apart
 *               (a multiple of 16 bytes), e.g. a slice of the projection
 *   conv_state  [batch, width-1, channels] x dtype (NULL for width 1)
 *   out         [batch, channels] x dtype, dense
 * channels a multiple of 8, width 1..8; x, conv_state, out 16-byte aligned. */
int ssd_causal_conv1d_step(const void *x, int64_t x_row_stride, void *conv_state,
                           const float *weight, const float *bias, int64_t batch,
                           int channels, int width, int silu, ssd_dtype_t dtype,
                           void *out, void *stream);

/* ---------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping by it:
 *   norm = sqrt(sum over tensors and elements of g^2)
 *   out  = g * min(1, max_norm / (norm + eps))
 * grads, sizes, dtypes, outs, out_dtypes are HOST arrays of `count` entries,
 * read during the call only: device addresses (aligned to their element),
 * element counts (0 allowed: the tensor is left out) and ssd_dtype_t values,
 * which may differ from tensor to tensor.  outs NULL: in place; else each
 * tensor's clipped values go to its own output, of out_dtypes (NULL: the
 * gradient's own type).  Tensors must not overlap one another.
 * norm: one float on the device (written).  Squares are summed in fp32 within
 * a chunk and in double beyond it, and in double throughout where a square
 * would leave the fp32 range; the factor takes the norm in double, so a finite
 * one that is infinite in *norm still scales.  A norm that is not finite is not
 * special: an infinite one gives the factor 0 (and NaN where g is infinite), a
 * NaN one gives NaN everywhere.  count may be 0 (norm = 0).  max_norm, eps >= 0. */
size_t ssd_clip_grads_workspace_bytes(int count);
int ssd_grad_norm(const void *const *grads, const int64_t *sizes,
                  const int32_t *dtypes, int count, float *norm,
                  void *workspace, size_t workspace_bytes, void *stream);
int ssd_clip_grads(const void *const *grads, const int64_t *sizes,
                   const int32_t *dtypes, int count, void *const *outs,
                   const int32_t *out_dtypes, float max_norm, float eps,
                   float *norm, void *workspace, size_t workspace_bytes,
                   void *stream);

/* ---------------------------------------------------------------------------
 * Projection with bias, activation and residual in one pass:
 *   pre = x W^T + bias,   out = act(pre) + residual
 *   x         [rows, in_features] x dtype, rows x_row_stride elements apart
 *   weight    [out_features, in_features] x dtype, dense
 *   bias      [out_features] x dtype, or NULL
 *   residual  [rows, out_features] fp32 or x dtype (residual_dtype), rows
 *             residual_row_stride elements apart, or NULL
 *   out       [rows, out_features] dense, of the residual's type, or the x
 *             dtype without one (written; may be the residual if it is dense,
 *             and must not overlap anything else)
 *   pre       [rows, out_features] dense, or NULL: the value before act, which
 *             the backward of an activation reads.  For bf16 it is kept in
 *             IEEE half (11 bits in the same 2 bytes: act' depends on pre by
 *             its absolute value only, so the half's range is enough: beyond
 *             it both activations are flat), for fp32 in fp32.
 * Sums in fp32 (bf16 products on the tensor cores; fp32 operands are split
 * into three bf16 parts each and their six leading products summed, about
 * fp32 accuracy for operands above 2^-110 in magnitude, whose third part is
 * still a normal bf16; a result within 2^-7 of the largest fp32 value may
 * come out infinite).  Infinities and NaN of an operand give the infinities and
 * NaN of the product in IEEE arithmetic.  SSD_ACT_GELU is v * Phi(v).
 * Any sizes and element-aligned pointers; bf16 operands whose rows are not all
 * 16-byte aligned (x, weight: in_features or the stride not a multiple of 8)
 * and fp32 ones are first laid out in the workspace.
 * The forward's workspace may be 0 bytes (workspace NULL): so it is where
 * operands are read where they lie and the sums are not split.
 * aligned (workspace queries): nonzero if x, weight (and for the backward dout)
 * are 16-byte aligned and x_row_stride is a multiple of 8.
 * rows <= 2^30, features <= 2^24.
 *
 * Backward for the upstream gradient dout of out ([rows, out_features] dense,
 * x dtype or fp32; also the residual's gradient, which needs no call):
 *   dpre = dout * act'(pre),  dx = dpre W,  dweight = dpre^T x,
 *   dbias = sum_rows dpre
 * dx [rows, in_features], dweight [out_features, in_features], dbias
 * [out_features], each x dtype, dense, or NULL (not computed); all written,
 * not accumulated.  For bf16, dpre is rounded to bf16 for the two products
 * (their operands' type) but not for dbias.
 * dout_as_is (workspace query): nonzero if there is no activation and dout has
 * the x dtype.  A wait inside the product kernel is bounded; ssd_scan_status
 * tells whether one gave up.
 * ------------------------------------------------------------------------- */
typedef enum { SSD_ACT_NONE = 0, SSD_ACT_SILU = 1, SSD_ACT_GELU = 2 } ssd_activation_t;

size_t ssd_linear_fwd_workspace_bytes(int64_t rows, int in_features,
                                      int out_features, ssd_dtype_t dtype,
                                      int aligned);
int ssd_linear_fwd(const void *x, int64_t x_row_stride, const void *weight,
                   const void *bias, const void *residual,
                   int64_t residual_row_stride, int64_t rows, int in_features,
                   int out_features, ssd_activation_t activation,
                   ssd_dtype_t dtype, ssd_dtype_t residual_dtype, void *out,
                   void *pre, void *workspace, size_t workspace_bytes,
                   void *stream);
size_t ssd_linear_bwd_workspace_bytes(int64_t rows, int in_features,
                                      int out_features, ssd_dtype_t dtype,
                                      int aligned, int dout_as_is);
int ssd_linear_bwd(const void *dout, ssd_dtype_t dout_dtype, const void *x,
                   int64_t x_row_stride, const void *weight, const void *pre,
                   int64_t rows, int in_features, int out_features,
                   ssd_activation_t activation, ssd_dtype_t dtype, void *dx,
                   void *dweight, void *dbias, void *workspace,
                   size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_BLOCK_H */
