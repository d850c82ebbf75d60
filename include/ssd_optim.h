/*
 * ssd_optim.h -- C ABI of the optimizer step that ends a training step (GB300,
 * sm_103a), after ssd_block.h's gradient norm: AdamW over many tensors at once,
 * with the moments in fp32 or in 8 bits.
 *
 * Conventions are those of ssd_scan.h and of ssd_clip_grads: arrays of `count`
 * entries are HOST arrays, read during the call only; they hold device addresses
 * (aligned to their element), element counts (0 allowed: the tensor is left out)
 * and ssd_dtype_t values.  Tensors must not overlap one another.  No atomics:
 * equal inputs give equal bits.
 */
#ifndef SSD_OPTIM_H
#define SSD_OPTIM_H

#include "ssd_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_OPTIM_ABI_VERSION 1
int ssd_optim_abi_version(void);

/* Values that share a scale of the 8-bit moments: block b of a tensor holds its
 * elements 256 b .. 256 b + 255. */
#define SSD_ADAMW_BLOCK 256

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;            /* number of this step, from 1 */
    const int64_t *step_dev; /* device: read instead of step where not NULL */
    const float *lr_dev;     /* device: read instead of lr where not NULL */
    const float *grad_norm;  /* device: the gradients' norm (ssd_grad_norm), or NULL: no clipping */
    double max_norm;
    uint32_t seed;           /* of the rounding of 8-bit moments */
} ssd_adamw_t;

/* One step of AdamW, in place, for each element of each tensor:
 *   g' = g * min(1, max_norm / (grad_norm + 1e-6))      (with grad_norm)
 *   m = beta1 m + (1 - beta1) g',   v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32 (g' too: not rounded to the gradients' type, as where ssd_clip_grads writes
 * it).  The factor keeps its bits where it is below the normal fp32 range; a norm that
 * is infinite in fp32 makes it 0, a NaN one makes everything NaN.  params, grads: fp32 or bf16, each tensor of its own dtype.  masters
 * NULL, or an array whose entry is NULL or the parameter's fp32 master: the step
 * is then the master's, and the parameter its rounded copy.
 * bits 32: exp_avgs, exp_avg_sqs are float, the scales NULL.
 * bits 8: codes, int8 for m and uint8 for v, with a float scale per block of
 * SSD_ADAMW_BLOCK elements (the largest |m|, v of the block):
 *   m = sign(c) (c / 127)^2 scale,   v = (c / 255)^4 scale
 * A new value lies between two codes and takes either, with the odds that keep
 * its mean (without that, an average with beta2 = 0.999 would stop moving: its
 * steps are smaller than half a code's); the random numbers are a hash of seed,
 * step, the tensor's number and the element's, so that equal calls give equal
 * codes.  A v above 0 keeps a code above 0.  A gradient that is not finite makes
 * its whole block's moments so.  The update itself takes m and v before they are
 * rounded to codes. */
int ssd_adamw_step(void *const *params, const int32_t *param_dtypes,
                   const void *const *grads, const int32_t *grad_dtypes,
                   float *const *masters, void *const *exp_avgs,
                   void *const *exp_avg_sqs, float *const *exp_avg_scales,
                   float *const *exp_avg_sq_scales, const int64_t *sizes,
                   int count, int bits, const ssd_adamw_t *options,
                   void *stream);

/* The values that 8-bit moments stand for, as fp32 tensors of their sizes. */
int ssd_adamw_moments(const void *const *exp_avgs, const void *const *exp_avg_sqs,
                      const float *const *exp_avg_scales,
                      const float *const *exp_avg_sq_scales,
                      float *const *exp_avg_values, float *const *exp_avg_sq_values,
                      const int64_t *sizes, int count, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_OPTIM_H */
