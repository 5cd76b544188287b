/*
 * nvfp4_block.h -- C ABI of a feed-forward block on MXFP4 operands and of its update (part of
 * libnvfp4.so): the FP4 product with bias, activation and residual in its epilogue, the gated
 * product, the activations' backward passes with the bias gradient, and AdamW over many tensors
 * with moments in 32 or 8 bits.
 *
 * Pointers, streams, workspaces and status codes follow nvfp4.h, element types, strides and
 * alignment nvfp4_train.h: device pointers of the caller, work enqueued on `stream`, argument
 * errors found before anything is enqueued, nothing allocated, nothing kept from call to call,
 * nothing copied to the host, each output rounded once.  Calls are safe under graph capture.  Results
 * do not depend on the order in which workgroups run.  Outputs must not overlap inputs, each
 * other or the workspace unless said.
 */
#ifndef NVFP4_BLOCK_H
#define NVFP4_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "nvfp4.h"
#include "nvfp4_train.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_ACT_NONE 0
#define NVFP4_ACT_RELU 1
#define NVFP4_ACT_GELU 2        /* z Phi(z) */
#define NVFP4_ACT_GELU_TANH 3   /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
#define NVFP4_ACT_SILU 4        /* z / (1 + e^-z) */

/* The product of two MXFP4 operands (nvfp4.h) with what follows it in a linear layer:
 *   z = f A B^T + bias,  y = act(z) + residual;                   gated 0
 *   z = (gate, up) = f A B^T + bias,  y = act(gate) up.           gated 1
 * a is [M][K], b [n][K] (gated: [2n][K], the gate's rows, then up's), both row-major or both
 * K-tiled; f = 2^-7 when rotated_pair != 0 (as for mxfp4_gemm) else 1.  Products are exact and
 * summed in FP32, in ascending 64-element steps of K or, with few rows, in a fixed order of
 * such sums.  bias [n] or [2n] (bias_type: `type` or F32) and residual [M][n] (`type`, row stride
 * residual_stride; not with gated) may be NULL.  y [M][n] and z [M][n] or [M][2n] (NULL: not kept),
 * contiguous, are of `type`; y comes from the unrounded z.  M, n >= 0, K a multiple of 128; sizes <
 * 2^31 (n < 2^30 where gated), products of two of them < 2^40. */
int mxfp4_linear_forward(const mxfp4_tensor *a, const mxfp4_tensor *b, int64_t M, int64_t n,
                         int64_t K, int rotated_pair, int gated, int activation, int type,
                         int bias_type, const void *bias, const void *residual,
                         int64_t residual_stride, void *y, void *z, void *stream);

/* Workspace bytes of activation_backward when dbias is wanted (16-byte aligned; 0 for few rows). */
size_t activation_backward_workspace_bytes(int type, int gated, int64_t rows, int64_t n);

/* The backward pass of y = act(z) (gated 0: z and dz [rows][n]) or of y = act(gate) up (gated 1: z
 * [rows][2n] holds gate, then up, and dz [rows][2n] their gradients) for dy [rows][n]:
 *   dz = dy act'(z);  dgate = dy up act'(gate),  dup = dy act(gate).
 * dy, z (row strides dy_stride, z_stride) and dz (contiguous) have one type.  dbias (bias_type: that
 * type or F32; may be NULL, then so may the workspace) is the sum of dz over the rows, [n] or [2n],
 * taken before dz is rounded.  relu'(0) is 0, and a relu's dz (or dgate) is 0 where z (or
 * gate) <= 0, whatever dy is.
 * z may be NULL for NVFP4_ACT_NONE without gating.  rows = 0 gives zeros in dbias.  Sizes and
 * strides < 2^31, products of rows with them < 2^40, n < 2^30 where gated. */
int activation_backward(int type, int bias_type, int activation, int gated, const void *dy,
                        int64_t dy_stride, const void *z, int64_t z_stride, int64_t rows,
                        int64_t n, void *dz, void *dbias, void *workspace,
                        size_t workspace_bytes, void *stream);

/* One parameter of adamw_step.  `param` and `grad` hold size < 2^40 adjacent elements of `type`
 * (NVFP4_F32, _BF16, _F16).  bits 32: m and v are float [size].  bits 8: m and v are codes
 * [blocks][128] (8-byte aligned) and m_scale and v_scale one byte a block, blocks =
 * ceil(size / 128); see below.  master (may be NULL; not with NVFP4_F32) is float [size]: the
 * parameter itself, of which `param` is the rounding to its type. */
typedef struct adamw_tensor {
    void *param;
    const void *grad;
    void *m;
    void *v;
    uint8_t *m_scale;
    uint8_t *v_scale;
    float *master;
    int64_t size;
    int32_t type;
    int32_t bits;
} adamw_tensor;

/* What adamw_step takes for all parameters together.  lr_device (float) and step_device
 * (int64_t) may be NULL; where given, they are read on `stream` in place of lr and step, so
 * that a captured call follows them.  norm (float, may be NULL) is the norm of all gradients:
 * they are taken times min(1, max_norm / (norm + 1e-6)), as clip_grads would scale them.  bounded: 1
 * or 0, of moments in 8 bits (see below). */
typedef struct adamw_options {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;
    const float *lr_device;
    const int64_t *step_device;
    const float *norm;
    float max_norm;
    int32_t bounded;
    uint64_t seed;
} adamw_options;

/* One AdamW step (Loshchilov and Hutter, decoupled weight decay) of `count` parameters, number
 * `step` >= 1 of their training:
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * in FP32.  tensors[] and *options are read on the host before the call returns.  0 <= beta1,
 * beta2 < 1; lr, eps and weight_decay >= 0 and finite.  A step_device below 1 counts as 1.
 *
 * Moments in 8 bits: m, and r = sqrt(v) in v's place, are rounded after the step that used them
 * unrounded.  A block of 128 elements has one power of two, scale byte s standing for 2^(s - 127):
 * the smallest that lets a code's largest value cover the block's (255: not a number in all of the
 * block, which a value that no power of two up to 2^126 covers makes it, such as an infinity or a
 * NaN; 0 belongs to zeros).  A code
 * is a floating number with four bits of exponent: r's has four bits of fraction, m's three and
 * the sign in bit 7; c = code without the sign, exponent field e, fraction f in [0, 1) stand for
 * (1 + f) 2^(e - 15), or f 2^-14 where e is 0.  Rounding is stochastic, so that what a moment
 * changes by, far less than a code's step, is not lost but kept on average: with 16 random bits u, the
 * magnitude's distance to the code below it, in steps, plus u 2^-16 is rounded down.  u is the upper
 * (m) or lower (r) half of word i mod 4 of Philox4x32-10 with the key `seed` at the counter (i / 4
 * lo, i / 4 hi, 2^31 + k, step lo), for element i of tensor k.  With `bounded` r's code is 1 at least
 * where r > 0.  Without, an r below 2^-18 of the block's power of two may become 0 where m does not, and the
 * next step divides m by its own gradient alone: where a block's gradients are spread over 10^5 and more
 * updates of several hundred lr were seen, with `bounded` none above 5 lr (32 bits: 1.4; beta1 0.9,
 * beta2 0.95 and 0.999, normal gradients).  A training run wants it.  All zeros are the moments before the
 * first step.  Elements of the last block past the parameter's end hold code 0. */
int adamw_step(const adamw_tensor *tensors, int64_t count, const adamw_options *options,
               void *stream);

/* The FP32 values [blocks][128] of 8-bit moments: codes [blocks][128] (8-byte aligned), one scale
 * byte a block; second 0 for m's codes, 1 for r's.  blocks < 2^33. */
int adamw_moment_values(const uint8_t *codes, const uint8_t *scales, int64_t blocks, int second,
                        float *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_BLOCK_H */
