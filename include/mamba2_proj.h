/*
 * mamba2_proj.h -- C ABI of the operators around a layer's projections: the norm
 * that takes the residual in, e4m3 values with power-of-two scales, and the matrix
 * product of such values; forward and backward.
 *
 * The conventions of mamba2_layer.h hold (device memory of the caller's, calls
 * asynchronous on `stream` and open to graph capture, argument errors before any
 * launch, token tensors with {batch, token} element strides, results that do not
 * depend on the order of blocks, calls that share a workspace must not overlap).
 *
 * Values in 8 bits.  A group of values is held as e4m3 numbers q (one byte each: sign,
 * 4 exponent bits, 3 mantissa bits, largest 448, no infinity) and one scale s = 2^e
 * (e8m0: the byte e + 127; 255 is NaN), of which they stand for q s.  Quantising takes the smallest
 * e >= -127 for which the group's largest magnitude is at most 448 * 2^e, and rounds x / s
 * to nearest even.  Infinities and NaN become NaN; the scale is that of the other values
 * (2^-127 in a group of zeros).  Groups are
 *   row:   128 neighbouring values of a row (the last of a row may be shorter): scales
 *          [.., ceil(D / 128)];
 *   block: 128 rows by 128 columns (shorter at the ends): scales [ceil(N / 128),
 *          ceil(K / 128)].
 * Rows of e4m3 values start on 16-byte boundaries: the address and the strides of such
 * a tensor are multiples of 16 (bytes behind a row's end are neither read nor written).
 */
#ifndef MAMBA2_PROJ_H
#define MAMBA2_PROJ_H

#include "mamba2_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- add_norm: RMS norm of the sum with the residual --------------------------
 *   total = x + residual, rounded to the residual's type (residual NULL: x)
 *   y = total w / sqrt(mean(total^2) + eps)          (w NULL: ones)
 * over the channels of each token.  y is io, or e4m3 in row groups with
 * MAMBA2_ADD_NORM_QUANT (rounded once, from fp32).  res_dtype, the type of residual and
 * total, is dtype or fp32.  channels at most 2^24, batch * seqlen below 2^31. */
#define MAMBA2_ADD_NORM_QUANT 1

typedef struct mamba2_add_norm_shape {
    int64_t batch, seqlen, channels;
    float eps;
    int32_t dtype;       /* mamba2_dtype of x and y */
    int32_t res_dtype;   /* mamba2_dtype of residual and total */
    int32_t flags;       /* MAMBA2_ADD_NORM_* */
} mamba2_add_norm_shape;

/* {batch, token} element strides; in the backward y is dy's and residual dtotal's. */
typedef struct mamba2_add_norm_strides {
    int64_t x[2], residual[2], y[2], total[2];
} mamba2_add_norm_strides;

/* x [b,T,D] io, residual [b,T,D] or NULL, w [D] fp32 or NULL -> y [b,T,D] (io or e4m3),
 * scales [b,T,ceil(D/128)] (with MAMBA2_ADD_NORM_QUANT, else NULL), total [b,T,D]. */
MAMBA2_API mamba2_status mamba2_add_norm_fwd(const mamba2_add_norm_shape* shape,
                                             const mamba2_add_norm_strides* strides,
                                             const void* x, const void* residual, const float* w,
                                             void* y, uint8_t* scales, void* total, void* stream);

/* Gradients for dL/dy = dy [b,T,D] io and dL/dtotal = dtotal [b,T,D] (of res_dtype, NULL =
 * 0), from the forward's total: dx [b,T,D] io, dresidual [b,T,D] of res_dtype (the same
 * values; NULL = not wanted), contiguous; dw [D] fp32 (NULL = not wanted).  A quantised
 * y's gradient is that of the values before rounding.  flags are ignored.  workspace:
 * mamba2_add_norm_bwd_workspace_size(shape) bytes, 16-byte aligned (partial sums of dw). */
MAMBA2_API size_t mamba2_add_norm_bwd_workspace_size(const mamba2_add_norm_shape* shape);
MAMBA2_API mamba2_status mamba2_add_norm_bwd(const mamba2_add_norm_shape* shape,
                                             const mamba2_add_norm_strides* strides,
                                             const void* total, const float* w, const void* dy,
                                             const void* dtotal, void* dx, void* dresidual, float* dw,
                                             void* workspace, size_t workspace_bytes, void* stream);

/* ---- quant8: values to e4m3 with scales ---------------------------------------
 * x [b,T,D] io -> q [b,T,D] e4m3, scales: row groups, or with MAMBA2_QUANT8_BLOCK (batch
 * 1: a weight [N, K] as seqlen N, channels K) block groups.  batch * seqlen below 2^31. */
#define MAMBA2_QUANT8_BLOCK 1

typedef struct mamba2_quant8_shape {
    int64_t batch, seqlen, channels;
    int32_t dtype;   /* mamba2_dtype of x */
    int32_t flags;   /* MAMBA2_QUANT8_* */
} mamba2_quant8_shape;

typedef struct mamba2_quant8_strides {
    int64_t x[2], q[2];
} mamba2_quant8_strides;

/* strides NULL: x contiguous, q's rows ceil(D / 16) * 16 apart. */
MAMBA2_API mamba2_status mamba2_quant8(const mamba2_quant8_shape* shape,
                                       const mamba2_quant8_strides* strides, const void* x,
                                       uint8_t* q, uint8_t* scales, void* stream);

/* ---- proj8: matrix product of values in 8 bits ---------------------------------
 *   y[m,n] = sum_k x[m,k] w[n,k]
 * x [tokens, inputs] e4m3 in row groups, w [outputs, inputs] e4m3 in block groups, sums in
 * fp32 on the tensor cores, y io.  Few tokens, and few tiles with long sums, split the sum
 * over a cluster of blocks (joined in a fixed order).  inputs >= 1; every size at most 2^30.
 * A wait for a copy, a product or another warp's work ends after two seconds: one that runs out
 * sets MAMBA2_DEVERR_TIMEOUT_PROJ8 in the word of mamba2_ssd_device_error, and the result is void.  A
 * cluster of blocks that comes to a stop so ends within six: those that wait for the one that gave up
 * take two more, what is in flight two at most.  (No limit of their own have the barriers at which a
 * cluster's blocks meet, which these waits lead to, the wait for the kernel before, and that for
 * tensor memory, which another stream's kernels may hold.) */
typedef struct mamba2_proj8_shape {
    int64_t tokens, inputs, outputs;
    int32_t dtype;   /* mamba2_dtype of y, dy and dx */
    int32_t flags;   /* 0 */
} mamba2_proj8_shape;

/* Elements between rows (pitches NULL: ceil(inputs / 16) * 16 for x and w, outputs for y), at
 * least a row's length; y also serves dy, whose rows may overlap (0: one row for all tokens). */
typedef struct mamba2_proj8_pitches {
    int64_t x, w, y;
} mamba2_proj8_pitches;

MAMBA2_API mamba2_status mamba2_proj8_fwd(const mamba2_proj8_shape* shape,
                                          const mamba2_proj8_pitches* pitches,
                                          const uint8_t* x, const uint8_t* x_scales,
                                          const uint8_t* w, const uint8_t* w_scales,
                                          void* y, void* stream);

/* Diagnostic: the failure path of these waits, without a fault.  Runs mamba2_proj8_fwd on tensors of
 * the default pitches with waits of `limit_us` microseconds (1 .. 100000), while one block of each
 * cluster keeps its scales back, for which the others then wait in vain.  The kernel returns
 * normally and the context stays usable; afterwards MAMBA2_DEVERR_TIMEOUT_PROJ8 is set, and y is
 * as it was. */
MAMBA2_API mamba2_status mamba2_proj8_selftest_timeout(const mamba2_proj8_shape* shape,
                                                       const uint8_t* x, const uint8_t* x_scales,
                                                       const uint8_t* w, const uint8_t* w_scales,
                                                       void* y, uint32_t limit_us, void* stream);

/* Gradients for dL/dy = dy [tokens, outputs] io: dx [tokens, inputs] io and dw [outputs,
 * inputs] fp32, contiguous; either may be NULL (not wanted).  Both products are taken in 8 bits:
 *   dx = Qrow(dy) w;   dw = Qcol(dy)^T Qcol(x)
 * where Qrow quantises in row groups and Qcol in groups of 128 tokens of one column (the
 * tokens 128 i .. 128 i + 127).  workspace: mamba2_proj8_bwd_workspace_size(shape) bytes,
 * 256-byte aligned (the quantised operands). */
MAMBA2_API size_t mamba2_proj8_bwd_workspace_size(const mamba2_proj8_shape* shape);
MAMBA2_API mamba2_status mamba2_proj8_bwd(const mamba2_proj8_shape* shape,
                                          const mamba2_proj8_pitches* pitches, const void* dy,
                                          const uint8_t* x, const uint8_t* x_scales,
                                          const uint8_t* w, const uint8_t* w_scales,
                                          void* dx, float* dw, void* workspace,
                                          size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_PROJ_H */
