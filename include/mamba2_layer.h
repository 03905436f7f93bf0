/*
 * mamba2_layer.h -- C ABI of the operators that stand around the chunked scan in
 * a layer: a short causal convolution, a selective scan with a decay per channel
 * and state, and a gated group norm; each forward and backward, and for single
 * tokens where it carries state.
 *
 * Conventions for every entry point.
 *   - All tensors are device memory owned by the caller; the library allocates
 *     nothing and keeps no state between calls.  Calls are asynchronous on
 *     `stream` (a cudaStream_t, NULL = the default stream) and may be captured
 *     into a CUDA graph; argument errors are returned before any launch.
 *   - "io" tensors hold `dtype` (fp32 or bf16); everything else is fp32.  All
 *     arithmetic is fp32; bf16 results are rounded once, to nearest even.
 *   - Token tensors are [batch, seqlen, width]: each token's `width` values are
 *     contiguous, and {batch, token} element strides are given by a strides
 *     struct (NULL = contiguous).  Inputs may have any strides >= 0 below 2^40;
 *     outputs must not overlap themselves.  Pointers need the alignment of their
 *     element type only; 16-byte aligned pointers and strides are faster.
 *   - Other tensors are contiguous.
 *   - `lengths` (device int32 [batch] or NULL): sequence i has lengths[i] tokens
 *     (clamped to 0 .. seqlen), the rest of its row is padding.  Padding is never
 *     part of a result whatever it holds (NaN and infinities included): outputs
 *     and gradients there are 0, and states are those after the last real token.
 *     A sequence of length 0 leaves its state as it came.
 *   - Outputs must not overlap inputs, except `state` of the step calls, which
 *     is updated in place.
 *   - Results do not depend on the order in which blocks run: sums over blocks are
 *     taken in a fixed order.  Calls that share a workspace must not overlap.
 *   - A zero batch or channel count is a no-op (gradients of parameters are
 *     written as 0); seqlen 0 copies the initial state to the final state.
 */
#ifndef MAMBA2_LAYER_H
#define MAMBA2_LAYER_H

#include "mamba2_ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- conv: short causal depthwise convolution over tokens -------------------
 *   s[b,t,c] = bias[c] + sum_{k < W} w[c,k] x[b, t - (W-1) + k, c]
 *   y        = s, or s * sigmoid(s) with MAMBA2_CONV_SILU
 * x before token 0 comes from initial_state (the W - 1 tokens before the first,
 * oldest first; NULL = 0); final_state holds the last W - 1 tokens seen.
 * width W in {2, 3, 4}. */
#define MAMBA2_CONV_SILU 1

typedef struct mamba2_conv_shape {
    int64_t batch, seqlen, channels;
    int32_t width;
    int32_t dtype;   /* mamba2_dtype */
    int32_t flags;   /* MAMBA2_CONV_* */
} mamba2_conv_shape;

/* {batch, token} element strides; y also serves dy in the backward. */
typedef struct mamba2_conv_strides {
    int64_t x[2], y[2];
} mamba2_conv_strides;

/* x [b,T,D] io, w [D,W], bias [D] or NULL, initial_state [b,W-1,D] io or NULL,
 * lengths or NULL -> y [b,T,D] io, final_state [b,W-1,D] io or NULL (not wanted). */
MAMBA2_API mamba2_status mamba2_conv_fwd(const mamba2_conv_shape* shape,
                                         const mamba2_conv_strides* strides,
                                         const void* x, const float* w, const float* bias,
                                         const void* initial_state, const int32_t* lengths,
                                         void* y, void* final_state, void* stream);

/* One token per sequence (seqlen 1): state [b,W-1,D] io, read and moved on by one
 * token in place; x, y [b,D] io (strides: the batch entries). */
MAMBA2_API mamba2_status mamba2_conv_step(const mamba2_conv_shape* shape,
                                          const mamba2_conv_strides* strides,
                                          void* state, const void* x, const float* w,
                                          const float* bias, void* y, void* stream);

/* Gradients of a loss with dL/dy = dy [b,T,D] io and dL/dfinal_state = dfinal
 * [b,W-1,D] io (NULL = 0).  Outputs: dx [b,T,D] io, dw [D,W] fp32, dbias [D] fp32
 * (NULL = not wanted), dinit [b,W-1,D] io (NULL = not wanted).  workspace:
 * mamba2_conv_bwd_workspace_size(shape) bytes, 16-byte aligned (partial sums of
 * dw and dbias). */
MAMBA2_API size_t mamba2_conv_bwd_workspace_size(const mamba2_conv_shape* shape);
MAMBA2_API mamba2_status mamba2_conv_bwd(const mamba2_conv_shape* shape,
                                         const mamba2_conv_strides* strides,
                                         const void* x, const float* w, const float* bias,
                                         const void* initial_state, const void* dy,
                                         const void* dfinal, const int32_t* lengths,
                                         void* dx, float* dw, float* dbias, void* dinit,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* ---- scan: selective scan with a decay per channel and state ----------------
 *   d_t = dt_t + dt_bias, or its softplus with MAMBA2_SCAN_SOFTPLUS
 *   h_t[c,n] = exp(d_t[c] A[c,n]) h_{t-1}[c,n] + d_t[c] x_t[c] B_t[g,n]
 *   y_t[c]   = sum_n C_t[g,n] h_t[c,n] + D[c] x_t[c],   times silu(z_t[c]) if z
 * Channel c reads group g = c / (channels / groups).  h_{-1} = initial_state
 * [b,D,N] (NULL = 0); final_state is h after the last token.  States are fp32.
 * states N in {8, 16, 32, 64, 128}; channels % groups == 0; groups * states and
 * channels at most 2^24, seqlen and batch at most 2^30. */
#define MAMBA2_SCAN_SOFTPLUS 1

typedef struct mamba2_scan_shape {
    int64_t batch, seqlen, channels, states, groups;
    int32_t dtype;   /* mamba2_dtype */
    int32_t flags;   /* MAMBA2_SCAN_* */
} mamba2_scan_shape;

/* {batch, token} element strides; y also serves dy in the backward. */
typedef struct mamba2_scan_strides {
    int64_t x[2], dt[2], B[2], C[2], z[2], y[2];
} mamba2_scan_strides;

/* x, dt [b,T,D] io, A [D,N], B, C [b,T,G,N] io, D [D] or NULL, z [b,T,D] io or
 * NULL, dt_bias [D] or NULL, initial_state [b,D,N] or NULL, lengths or NULL
 * -> y [b,T,D] io, final_state [b,D,N].  workspace: mamba2_scan_workspace_size(
 * shape) bytes (may be 0), 16-byte aligned, contents ignored on entry: with few rows
 * the states between the stretches of tokens that run side by side; with more rows
 * than the GPU holds at once, which then take turns in slices of the token axis, one
 * word a row (a slice waits for the slice before it, at most two seconds).  A wait that
 * runs out sets MAMBA2_DEVERR_CHAIN_SCAN in the word of mamba2_ssd_device_error and gives
 * the row up: its slices from there on leave at once, y is not written there, and
 * final_state is not the row's last state. */
MAMBA2_API size_t mamba2_scan_workspace_size(const mamba2_scan_shape* shape);
MAMBA2_API mamba2_status mamba2_scan_fwd(const mamba2_scan_shape* shape,
                                         const mamba2_scan_strides* strides,
                                         const void* x, const void* dt, const float* A,
                                         const void* B, const void* C, const float* D,
                                         const void* z, const float* dt_bias,
                                         const float* initial_state, const int32_t* lengths,
                                         void* y, float* final_state,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* Diagnostic: the failure path of the wait described above, without a fault.  Runs
 * mamba2_scan_fwd on contiguous tensors with the first slice of tokens launched after all
 * the others, whose waits run out after `limit_us` microseconds (1 .. 100000).  All
 * launches return normally and the context stays usable; afterwards
 * MAMBA2_DEVERR_CHAIN_SCAN is set, y holds the first slice only, and the workspace's word
 * of every row is -1 (given up; the late first slice does not take that back).  Returns
 * MAMBA2_ERR_UNSUPPORTED for a shape whose rows do not take turns. */
MAMBA2_API mamba2_status mamba2_scan_selftest_turn_timeout(const mamba2_scan_shape* shape,
                                                           const void* x, const void* dt, const float* A,
                                                           const void* B, const void* C, void* y,
                                                           float* final_state, void* workspace,
                                                           size_t workspace_bytes, uint32_t limit_us,
                                                           void* stream);

/* One token per sequence (seqlen 1): state [b,D,N] fp32 updated in place; x, dt,
 * z, y [b,D] and B, C [b,G,N] io (strides: the batch entries). */
MAMBA2_API mamba2_status mamba2_scan_step(const mamba2_scan_shape* shape,
                                          const mamba2_scan_strides* strides,
                                          float* state, const void* x, const void* dt,
                                          const float* A, const void* B, const void* C,
                                          const float* D, const void* z, const float* dt_bias,
                                          void* y, void* stream);

/* Gradients of a loss with dL/dy = dy [b,T,D] io and dL/dfinal_state = dfinal
 * [b,D,N] (NULL = 0), recomputing the forward's states.  Outputs: dx, ddt (of dt
 * as given, before the bias) [b,T,D], dz (required when z is given) [b,T,D], dB,
 * dC [b,T,G,N], all io and contiguous; dA [D,N], dD [D] (required when D is
 * given), ddt_bias [D] (required when dt_bias is given), dinit [b,D,N] (NULL =
 * not wanted), fp32. */
MAMBA2_API size_t mamba2_scan_bwd_workspace_size(const mamba2_scan_shape* shape);
MAMBA2_API mamba2_status mamba2_scan_bwd(const mamba2_scan_shape* shape,
                                         const mamba2_scan_strides* strides,
                                         const void* x, const void* dt, const float* A,
                                         const void* B, const void* C, const float* D,
                                         const void* z, const float* dt_bias,
                                         const float* initial_state, const void* dy,
                                         const float* dfinal, const int32_t* lengths,
                                         void* dx, void* ddt, float* dA, void* dB, void* dC,
                                         float* dD, void* dz, float* ddt_bias, float* dinit,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* ---- norm: RMS norm over groups of channels, with a SiLU gate ---------------
 * Per token and group of S = channels / groups channels:
 *   gate first: v = x silu(z);  y = v w / sqrt(mean_S(v^2) + eps)
 *   gate after (MAMBA2_NORM_GATE_AFTER): y = x w / sqrt(mean_S(x^2) + eps) silu(z)
 * z NULL: no gate.  w NULL: ones.  A row of zeros gives zeros (eps > 0). */
#define MAMBA2_NORM_GATE_AFTER 1

typedef struct mamba2_norm_shape {
    int64_t batch, seqlen, channels, groups;
    float eps;
    int32_t dtype;   /* mamba2_dtype */
    int32_t flags;   /* MAMBA2_NORM_* */
} mamba2_norm_shape;

/* {batch, token} element strides; y also serves dy in the backward. */
typedef struct mamba2_norm_strides {
    int64_t x[2], z[2], y[2];
} mamba2_norm_strides;

/* x [b,T,D] io, w [D] or NULL, z [b,T,D] io or NULL -> y [b,T,D] io. */
MAMBA2_API mamba2_status mamba2_norm_fwd(const mamba2_norm_shape* shape,
                                         const mamba2_norm_strides* strides,
                                         const void* x, const float* w, const void* z,
                                         void* y, void* stream);

/* Gradients for dL/dy = dy [b,T,D] io: dx, dz (required when z is given) [b,T,D]
 * io, contiguous; dw [D] fp32 (NULL = not wanted).  workspace:
 * mamba2_norm_bwd_workspace_size(shape) bytes, 16-byte aligned (partial sums of dw). */
MAMBA2_API size_t mamba2_norm_bwd_workspace_size(const mamba2_norm_shape* shape);
MAMBA2_API mamba2_status mamba2_norm_bwd(const mamba2_norm_shape* shape,
                                         const mamba2_norm_strides* strides,
                                         const void* x, const float* w, const void* z,
                                         const void* dy, void* dx, void* dz, float* dw,
                                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_LAYER_H */
