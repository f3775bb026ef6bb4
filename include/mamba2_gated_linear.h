/*
 * mamba2_gated_linear.h — C ABI of a recurrent block's operators on GB300
 * (sm_103a), for training and for serving: the gated linear recurrence (one
 * state value a channel) with its backward pass and its form for single
 * tokens, the norms after and before a block joined with its gate and the
 * residual sum, forward and backward, and the gradient of the causal
 * convolution of mamba2_gated_delta.h, which runs in front of the recurrence.
 *
 * The conventions of mamba2_ssd.h hold for every entry point: device pointers
 * owned by the caller, arguments checked on the host before anything is
 * launched, work enqueued on the caller's stream, nothing allocated, nothing
 * synchronised, every output fully overwritten, outputs overlap no input and
 * one another (except where said), statuses of mamba2_status.  fp32 weights,
 * their gradients, states and workspaces are aligned to 16 bytes; sequences and
 * rows, and their gradients, only to their element, so that slices of a wider
 * tensor can be passed with their token stride (16-byte aligned ones take the
 * faster loads; slices side by side in one tensor do not count as overlapping).
 * A gradient is the same for the same call: sums run in a fixed order.
 */
#ifndef MAMBA2_GATED_LINEAR_H
#define MAMBA2_GATED_LINEAR_H

#include "mamba2_gated_delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------- gated linear recurrence
 * Per batch row and channel:
 *
 *     log a_t = A sigmoid(r_t)
 *     h_t     = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
 *     y_t     = h_t, or h_t SiLU(z_t) with z
 *
 *   x, r, i, z, y [b, L, C]   dtype   r, i, z before their activations; z may be NULL
 *   A             [C]         fp32    log decay at an open gate, <= 0 (not checked)
 *   initial_state, final_state [b, C] fp32 (NULL: zeros; not written)
 *   chunk_states  [b, nc, C]  fp32    h before token 64 k, nc = ceil(L / 64): what
 *                                     the backward pass starts from (NULL: not written)
 *   lengths       [b]         int32, NULL means L for every row
 *
 * With lengths, row b has min(max(lengths[b], 0), L) tokens: y is 0 past them,
 * final_state (and chunk_states past them) the state after them, and nothing
 * there is read into a result.  Gates and states are fp32 for both dtypes.
 * r_t = -infinity keeps the state (to fp32's rounding).  At most 65535 batch
 * rows, 2^30 tokens, 2^30 channels and 2^33 states of all batch rows; tensors of
 * more than 2^40 elements, strides included, are MAMBA2_ERR_UNSUPPORTED, too. */
enum { MAMBA2_GLR_CHUNK = 64 };

typedef struct {
    int64_t batch, seqlen, channels;
    int64_t x_stride, r_stride, i_stride; /* elements from token to token (0: channels) */
    int64_t z_stride, y_stride;           /* (the backward pass: y_stride is dy's) */
    int32_t dtype;                        /* mamba2_dtype */
    int32_t flags;                        /* must be 0 */
} mamba2_glr_shape;

MAMBA2_API mamba2_status mamba2_glr_fwd(const mamba2_glr_shape* shape, const void* x, const void* r, const void* i,
                                        const void* z, const float* A, const int32_t* lengths,
                                        const float* initial_state, void* y, float* chunk_states, float* final_state,
                                        struct CUstream_st* stream);

/* Gradients of a forward call with the same shape, inputs and lengths, whose
 * chunk_states are given.  dy [b, L, C] dtype; dfinal_state [b, C] fp32 (NULL:
 * zeros).  dx, dr, di (and dz with z, else NULL) [b, L, C] dtype, 0 past a row's
 * length; dA [C] fp32 (not a number where A is 0, where it has no value);
 * dinitial_state [b, C] fp32 (NULL: not written).  grad_strides: elements from
 * token to token of dx, dr, di, dz (0: channels; NULL: all 0).  workspace:
 * mamba2_glr_bwd_workspace_size(shape) bytes, aligned to 256, used by this call
 * only. */
typedef struct {
    int64_t dx_stride, dr_stride, di_stride, dz_stride;
} mamba2_glr_grad_strides;

MAMBA2_API size_t mamba2_glr_bwd_workspace_size(const mamba2_glr_shape* shape); /* 0 for a bad shape */
MAMBA2_API mamba2_status mamba2_glr_bwd(const mamba2_glr_shape* shape, const mamba2_glr_grad_strides* grad_strides,
                                        const void* dy, const void* x, const void* r, const void* i, const void* z,
                                        const float* A, const int32_t* lengths, const float* chunk_states,
                                        const float* dfinal_state, void* dx, void* dr, void* di, void* dz, float* dA,
                                        float* dinitial_state, void* workspace, size_t workspace_bytes,
                                        struct CUstream_st* stream);

/* One token (shape->seqlen must be 1): strides go from one batch row to the
 * next; state_in NULL means zeros; state_out is required and may be the same
 * pointer as state_in (update in place). */
MAMBA2_API mamba2_status mamba2_glr_step(const mamba2_glr_shape* shape, const void* x, const void* r, const void* i,
                                         const void* z, const float* A, const float* state_in, float* state_out,
                                         void* y, struct CUstream_st* stream);

/* ------------------------------------- gradient of the causal convolution
 * Of mamba2_causal_conv_fwd with the same shape (whose y_stride is dy's here)
 * and inputs: dx [b, L, C] dtype (dx_stride 0: channels; 0 past a row's length,
 * where dy is not read), dweight [C, W] and dbias [C] fp32 (dbias NULL: not
 * written), dinitial_state [b, W - 1, C] dtype (NULL: not written).
 * dfinal_state [b, W - 1, C] dtype (NULL: zeros) is the gradient of final_state.
 * workspace: mamba2_causal_conv_bwd_workspace_size(shape) bytes, aligned to 256. */
MAMBA2_API size_t mamba2_causal_conv_bwd_workspace_size(const mamba2_conv_shape* shape); /* 0 for a bad shape */
MAMBA2_API mamba2_status mamba2_causal_conv_bwd(const mamba2_conv_shape* shape, int64_t dx_stride, const void* dy,
                                                const void* x, const float* weight, const float* bias,
                                                const int32_t* lengths, const void* initial_state,
                                                const void* dfinal_state, void* dx, float* dweight, float* dbias,
                                                void* dinitial_state, void* workspace, size_t workspace_bytes,
                                                struct CUstream_st* stream);

/* ------------------------------------------- norms after and before a block
 * Per row (token), with N(v) = v / sqrt(mean(v^2) + eps) over the row's channels:
 *
 *     p            = x, or post_weight N(x) with MAMBA2_BLOCK_NORM_POST
 *     p            = p SiLU(z)                                   with z
 *     residual_out = residual + scale p
 *     y            = pre_weight N(residual_out)                  with MAMBA2_BLOCK_NORM_PRE
 *
 *   x, z, y      [rows, channels] dtype: the block's output, its gate (NULL: none), the
 *                next block's input (with PRE, else NULL)
 *   residual     [rows, channels] residual_dtype (NULL: zeros)
 *   residual_out [rows, channels] residual_dtype; may be the same pointer as residual
 *                (with the same stride): updated in place
 *   post_weight, scale, pre_weight [channels] fp32; NULL means 1
 * Sums in fp32: a row whose sum of squares passes fp32's largest number has N = 0, and
 * passes no gradient through it.  y comes from the sum before it is rounded to
 * residual_dtype, which is no narrower than dtype (else MAMBA2_ERR_UNSUPPORTED).  At
 * most 32768 channels, fewer than 2^31 rows, rows x stride up to 2^40. */
enum { MAMBA2_BLOCK_NORM_POST = 1, MAMBA2_BLOCK_NORM_PRE = 2 };

typedef struct {
    int64_t rows, channels;
    int64_t x_stride, z_stride;                        /* elements from row to row (0: channels) */
    int64_t residual_stride, residual_out_stride;
    int64_t y_stride;                                  /* (the backward pass: dy's) */
    float eps;                                         /* > 0 */
    int32_t dtype, residual_dtype;                     /* mamba2_dtype */
    int32_t flags;
} mamba2_block_norm_shape;

MAMBA2_API mamba2_status mamba2_block_norm_fwd(const mamba2_block_norm_shape* shape, const void* x, const void* z,
                                               const void* residual, const float* post_weight, const float* scale,
                                               const float* pre_weight, void* residual_out, void* y,
                                               struct CUstream_st* stream);

/* Its gradients, from x, z, the weights and (with PRE) residual_out as the
 * forward call wrote it: dresidual_out [rows, channels] residual_dtype (NULL:
 * zeros) and dy [rows, channels] dtype (with PRE, else NULL) come in; dx, dz (with
 * z, else NULL) dtype, dresidual residual_dtype (NULL: not written; may be the
 * same pointer as dresidual_out, with the same stride), and dpost_weight, dscale,
 * dpre_weight [channels] fp32 (NULL: not written; dpost_weight only with POST,
 * dpre_weight only with PRE) go out.  shape's residual_stride is not used.  grad_strides: elements from row
 * to row (0: channels; NULL: all 0).  workspace:
 * mamba2_block_norm_bwd_workspace_size(shape) bytes, aligned to 256. */
typedef struct {
    int64_t dx_stride, dz_stride, dresidual_out_stride, dresidual_stride;
} mamba2_block_norm_grad_strides;

MAMBA2_API size_t mamba2_block_norm_bwd_workspace_size(const mamba2_block_norm_shape* shape); /* 0: bad shape */
MAMBA2_API mamba2_status mamba2_block_norm_bwd(const mamba2_block_norm_shape* shape,
                                               const mamba2_block_norm_grad_strides* grad_strides,
                                               const void* dresidual_out, const void* dy, const void* x,
                                               const void* z, const void* residual_out, const float* post_weight,
                                               const float* scale, const float* pre_weight, void* dx, void* dz,
                                               void* dresidual, float* dpost_weight, float* dscale,
                                               float* dpre_weight, void* workspace, size_t workspace_bytes,
                                               struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_GATED_LINEAR_H */
