/*
 * wtconv_optim.h -- AdamW over many tensors and the global gradient norm, part of libwtconv.so
 * (GB300, sm_103a).
 *
 * One call updates every tensor of a model, of any sizes:
 *
 *     g' = clip g,   m' = beta1 m + (1 - beta1) g',   v' = beta2 v + (1 - beta2) g'^2
 *     p' = p (1 - lr weight_decay) - lr / (1 - beta1^t) m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
 *
 * Parameters are fp32 (as everywhere in this library); gradients fp32, bf16 or fp16; a 16-bit
 * working copy of the parameters can be written in the same pass.  All arithmetic is fp32.
 *
 * States m, v in 32 bits, or in 8: blocks of WTCONV_ADAMW_BLOCK elements of a tensor share the
 * maxima M of |m| and of v (fp32, one each per block, the last block may be short), and hold
 *
 *     m = c |c| / 127^2 M   (c a signed byte),      v = (c / 255)^4 M   (c an unsigned byte)
 *
 * whose steps shrink towards zero with the value.  A new value lies between the values of two
 * neighbouring codes, at a share s of the way; it takes the upper one if s > u, with
 * u = frac((i K1 + t K2) / 2^32) from the element's index i in its tensor and the step number t
 * (K1, K2 = 2^32 / p, 2^32 / p^2, p^3 = p + 1: u is spread evenly over neighbours and over steps).
 * On average over steps the rounding so cancels: v moves by 1 - beta2 = 0.1 % a step, far less
 * than the distance of two codes, and would stand still if it went to the nearest code.  A
 * positive v never takes code 0 (sqrt(v) divides).  A block whose maximum is below 2^-90 is held
 * as zeros.
 *
 * Non-finite values: where *clip is not finite (see wtconv_grad_norm) the call leaves every tensor
 * as it is.  Without clip, a non-finite gradient makes its element's p, m and v non-finite (with
 * 8-bit states: the m and v of its block).  A finite one whose square passes fp32 (above 1.8e19)
 * makes its v infinite; in 8 bits that leaves its block's v infinite or NaN, and from the next step
 * on the parameters under a NaN are NaN.  sqrt(v') is that of at least 2^-126.
 *
 * Conventions are those of wtconv.h: device pointers in a host array of descriptors (read before
 * the call returns), asynchronous on `stream`, nothing allocated, arguments checked before any
 * launch.  Pointers need only their element's alignment; tensors whose pointers are all 16-byte
 * aligned run fastest.  No two tensors' outputs may overlap (a shared parameter is given once).
 * Descriptors with n = 0 are skipped (their pointers may be NULL).  Results do not depend on how
 * tensors are grouped, except the last bits of the norm.
 */
#ifndef WTCONV_OPTIM_H
#define WTCONV_OPTIM_H

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WTCONV_ADAMW_BLOCK 256

/* One tensor of n elements.  m, v: float[n], or with 8-bit states int8[n], uint8[n] and the block
 * maxima m_max, v_max: float[ceil(n / 256)] (NULL with 32-bit states).  copy: 16-bit working copy
 * of the parameters, or NULL. */
typedef struct wtconv_optim_tensor {
    float *param;
    const void *grad;
    void *m, *v;
    float *m_max, *v_max;
    void *copy;
    long long n;
} wtconv_optim_tensor;

/* Scalars of a step.  step counts from 1. */
typedef struct wtconv_adamw_config {
    double lr, beta1, beta2, eps, weight_decay;
    long long step;
    int state_bits;  /* 32 or 8 */
    int grad_dtype;  /* enum wtconv_dtype */
    int copy_dtype;  /* WTCONV_BF16 or WTCONV_F16 where any copy is given; ignored otherwise */
} wtconv_adamw_config;

/* One AdamW step.  clip: device pointer to the gradients' factor, or NULL for 1.
 * 0 <= lr, eps, weight_decay; 0 <= beta1, beta2 < 1. */
int wtconv_adamw_step(int n_tensors, const wtconv_optim_tensor *tensors,
                      const wtconv_adamw_config *config, const float *clip, wtconv_stream_t stream);

/* Values of 8-bit states as fp32: m_out[i], v_out[i] (host arrays of device pointers, float[n])
 * from tensor i.  Either array may be NULL. */
int wtconv_adamw_state_values(int n_tensors, const wtconv_optim_tensor *tensors,
                              float *const *m_out, float *const *v_out, wtconv_stream_t stream);

/* Bytes of device workspace wtconv_grad_norm needs (16-byte aligned; 0 for few elements, which one
 * launch sums). */
size_t wtconv_grad_norm_workspace_size(int n_tensors, const wtconv_optim_tensor *tensors);

/* out[0] = norm = sqrt(sum of squares of every gradient), out[1] = the factor that limits it to
 * max_norm: min(1, max_norm / (norm + 1e-6)), or NaN where the norm is not finite.  out is device
 * memory that wtconv_adamw_step can take its clip from (out + 1), with no host in between.  Squares
 * are summed in fp32 over at most a few hundred elements of a thread and in fp64 beyond, in an order
 * that depends on the device and on the tensors' sizes and 16-byte alignment only; a gradient above
 * 1.8e19, whose square passes fp32, makes the norm infinite.  max_norm > 0 (infinity: the factor is
 * 1).  Reads only grad and n of each descriptor. */
int wtconv_grad_norm(int n_tensors, const wtconv_optim_tensor *tensors, int grad_dtype,
                     double max_norm, float *out, void *workspace, size_t workspace_bytes,
                     wtconv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_OPTIM_H */
