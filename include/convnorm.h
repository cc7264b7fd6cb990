/*
 * convnorm.h -- C ABI of the channels-last group norm of the convolution
 * library for AMD Instinct MI355X (gfx950): what stands between the
 * convolutions of convfwd.h, and after the heads of a sequence layer.
 *
 * x is (N, P, C), channels fastest: P positions of N images or volumes, or P =
 * 1 for rows that are normalised each.  Groups are C / groups neighbouring
 * channels.  Over the P * C / groups values of each (n, group), with the biased
 * variance,
 *
 *   xhat = (x - mean) * rstd,  rstd = 1 / sqrt(var + eps)
 *   z = xhat * weight[c] + bias[c],  y = z or z * sigmoid(z)
 *
 * dtype (convfwd_dtype) is the type of x, y and their gradients; weight and
 * bias have param_dtype, which is dtype or fp32.  mean, rstd and the gradients
 * of weight and bias are fp32.  All arithmetic is fp32 (the sums of tiles are
 * joined in fp64), results are rounded once, to nearest even, and sums are added
 * in a fixed order: the same call gives the same bits.  The variance is taken
 * about the mean where a group fits one workgroup's registers.  In larger groups
 * each channel's runs of r positions (8, or more of large tensors) take theirs
 * about their first value, which costs up to r times fp32's error where that
 * value is an outlier, and are joined about the mean: nothing depends on how far
 * the mean is from zero.
 *
 * An infinity or a NaN in a group makes the whole group NaN, as the formula
 * has it, and touches no other group; in the backward pass it also reaches the
 * gradients of the parameters of its channels.
 *
 * Inputs marked "rows" may be views as in convseq.h: channel stride 1, any
 * batch and position stride >= 0 (batch_stride, row_stride).  Everything else
 * is dense.  Ownership, streams, workspaces and errors are those of convseq.h.
 * N = 0 and P = 0 are valid: outputs over positions are empty, the mean of
 * nothing is 0 and its variance 0, gradients of parameters are zero.
 */
#ifndef CONVNORM_H
#define CONVNORM_H

#include <stdint.h>

#include "convseq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t n, p, c;
  int32_t groups;      /* divides c */
  int32_t act;         /* convseq_act */
  int32_t dtype;       /* convfwd_dtype */
  int32_t param_dtype; /* dtype or CONVFWD_F32 */
  float eps;           /* >= 0 */
} convnorm_desc;

/* y (N, P, C), mean and rstd (N, groups).  weight and bias (C) may be NULL: 1 and 0. */
int64_t convnorm_group_fwd_workspace(const convnorm_desc* desc); /* bytes, or a negative error */
int convnorm_group_fwd(const convnorm_desc* desc, const convseq_rows* x, const void* weight, const void* bias, void* y,
                       void* mean, void* rstd, void* workspace, void* stream);

/* Gradients of convnorm_group_fwd: dy (N, P, C) is that of y; x, weight, bias,
 * mean and rstd are the forward pass's.  dx (N, P, C); dweight and dbias (C),
 * fp32, may be NULL.  (mean and rstd are taken as functions of x: dx is the whole
 * gradient.) */
int64_t convnorm_group_bwd_workspace(const convnorm_desc* desc); /* bytes, or a negative error */
int convnorm_group_bwd(const convnorm_desc* desc, const convseq_rows* dy, const convseq_rows* x, const void* weight,
                       const void* bias, const void* mean, const void* rstd, void* dx, void* dweight, void* dbias,
                       void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVNORM_H */
