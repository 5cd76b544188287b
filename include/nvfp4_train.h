/*
 * nvfp4_train.h -- C ABI of the operators around the quantized linear layer in a training step
 * (part of libnvfp4.so): layer norm, softmax cross entropy of a linear head over a large
 * vocabulary, and the global gradient norm with clipping.
 *
 * Pointers, streams, workspaces and status codes follow nvfp4.h: device pointers of the caller,
 * work enqueued on `stream`, argument errors found before anything is enqueued, nothing
 * allocated, nothing kept from call to call, nothing copied to the host.  Calls are safe under
 * graph capture.  Results do not depend on the order in which workgroups run.
 *
 * Element types are NVFP4_F32, NVFP4_BF16 and NVFP4_F16.  Data pointers need their element's
 * alignment only.  Strides are in elements; a row's elements are adjacent.  Sums, statistics and
 * products are held in at least FP32 and each output is rounded once, except where said.
 * Outputs must not overlap inputs, each other or the workspace unless said.
 */
#ifndef NVFP4_TRAIN_H
#define NVFP4_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_F32 0
#define NVFP4_BF16 1
#define NVFP4_F16 2

#define NVFP4_SUM 0
#define NVFP4_MEAN 1
#define NVFP4_NONE 2

/* y = (x - mean) rstd weight + bias for each row of x [rows][n] (row stride x_stride >= n, n >=
 * 1), with mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps).  weight and bias [n]
 * may be NULL (1 and 0); they have the type p_type: x's type or F32.  y [rows][n] contiguous in
 * x's type, mean and rstd [rows] FP32.  eps >= 0 and finite.  rows, n and the strides < 2^31, rows
 * times n or a stride < 2^40. */
int layer_norm_forward(int type, int p_type, const void *x, const void *weight, const void *bias,
                       int64_t rows, int64_t n, int64_t x_stride, float eps, void *y,
                       float *mean, float *rstd, void *stream);

/* Workspace bytes of layer_norm_backward when dweight or dbias is wanted. */
size_t layer_norm_workspace_bytes(int type, int64_t rows, int64_t n);

/* dx [rows][n] (contiguous, x's type) and, where not NULL, dweight and dbias [n] (p_type) from
 * dy (row stride dy_stride) and the forward pass's x, mean, rstd and weight.  rows = 0 gives
 * zeros in dweight and dbias.  The workspace (16-byte aligned) may be NULL where neither is
 * wanted. */
int layer_norm_backward(int type, int p_type, const void *dy, const void *x, const float *mean,
                        const float *rstd, const void *weight, int64_t rows, int64_t n,
                        int64_t dy_stride, int64_t x_stride, void *dx, void *dweight,
                        void *dbias, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of the two calls below (256-byte aligned); backward 0 or 1. */
size_t linear_cross_entropy_workspace_bytes(int backward, int64_t t, int64_t d, int64_t v);

/* Cross entropy of the logits h w^T, h [t][d] and w [v][d] of one type (BF16 or F16), without
 * holding them: lse[i] = log sum exp of token i's logits and loss = lse - logit of target[i].
 * Tokens whose target is ignore_index do not count: their loss and lse are 0, and nothing in
 * their rows of h reaches a result.  A target outside [0, v) that is not ignore_index has the
 * loss NaN.  reduction NVFP4_NONE: loss [t]; NVFP4_SUM, NVFP4_MEAN (over the tokens that
 * count; 0 where none does): loss [1].  lse [t].  t, v < 2^28, d and the strides < 2^31, d >= 1, v
 * >= 1, each product of two sizes, or of a stride and its rows, < 2^40. */
int linear_cross_entropy_forward(int type, const void *h, int64_t h_stride, const void *w,
                                 int64_t w_stride, const int64_t *target, int64_t t, int64_t d,
                                 int64_t v, int64_t ignore_index, int reduction, float *loss,
                                 float *lse, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* Gradients dh [t][d] and dw [v][d] (contiguous, the inputs' type; either may be NULL) of the
 * loss above, whose gradient is dloss: [t] FP32 for NVFP4_NONE, [1] otherwise.  lse is the
 * forward pass's.  Rows of dh of tokens that do not count are 0.  A token with a target outside
 * the vocabulary makes its row of dh and all of dw NaN.  The softmax's gradient enters the two
 * products rounded to the inputs' type, of up to 128 tokens as the sum of two such numbers: before
 * dloss, which the FP32 results take, except in dw of NVFP4_NONE, whose sum is over tokens of
 * different dloss. */
int linear_cross_entropy_backward(int type, const float *dloss, const void *h, int64_t h_stride,
                                  const void *w, int64_t w_stride, const int64_t *target,
                                  const float *lse, int64_t t, int64_t d, int64_t v,
                                  int64_t ignore_index, int reduction, void *dh, void *dw,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of grad_norm and clip_grads (8-byte aligned) for `count` tensors of sizes[]
 * elements; 0 where a size is negative. */
size_t grad_norm_workspace_bytes(const int64_t *sizes, int64_t count);

/* norm[0] = sqrt of the sum of squares (inf = 0) or the largest magnitude (inf = 1) over all
 * elements of `count` tensors.  tensors[], sizes[] and types[] are HOST arrays, read before the
 * call returns; tensor i is sizes[i] < 2^40 adjacent elements of types[i].  A NaN anywhere makes
 * the norm NaN.  No tensors, or only empty ones, have the norm 0. */
int grad_norm(const void *const *tensors, const int64_t *sizes, const int32_t *types,
              int64_t count, int inf, float *norm, void *workspace, size_t workspace_bytes,
              void *stream);

/* grad_norm, then outs[i] = tensors[i] * min(1, max_norm / (norm + 1e-6)), each rounded to its
 * type; outs[i] is tensors[i] itself or does not overlap any tensor,
 * nor do two outs overlap (NVFP4_ERR_ARG).  max_norm >= 0.  Where the
 * factor is 1, tensors clipped in place are not written. */
int clip_grads(const void *const *tensors, void *const *outs, const int64_t *sizes,
               const int32_t *types, int64_t count, float max_norm, int inf, float *norm,
               void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_TRAIN_H */
