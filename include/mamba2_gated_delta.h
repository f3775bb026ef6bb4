/*
 * mamba2_gated_delta.h — C ABI of the gated-delta-rule layer's operators on
 * GB300 (sm_103a): the gated delta rule over whole sequences and one token at
 * a time, the short causal convolution that makes its inputs, and the group
 * norm with a gate or an activation that follows it.  The convolution and the
 * norm are also those on either side of the state-space recurrence of
 * mamba2_ssd.h.
 *
 * The conventions of mamba2_ssd.h hold for every entry point: device pointers
 * owned by the caller, arguments checked on the host before anything is
 * launched, work enqueued on the caller's stream, nothing allocated, nothing
 * synchronised, every output fully overwritten, outputs overlap no input
 * (except where said), statuses of mamba2_status.  Pointers are aligned to 16
 * bytes; q, k, v of the gated delta rule, the convolution's x and y and the
 * norm's x, z and y only to their element, so that slices of a wider tensor
 * can be passed with their token stride (16-byte aligned ones take the faster
 * loads).
 */
#ifndef MAMBA2_GATED_DELTA_H
#define MAMBA2_GATED_DELTA_H

#include "mamba2_ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- gated delta rule
 * Per batch row and head, with a state h of S x H (state rows x head dim):
 *
 *     h_t = e^{g_t} h_{t-1} + k_t (beta_t (v_t - (e^{g_t} h_{t-1})^T k_t))^T
 *     y_t = scale h_t^T q_t
 *
 * The state first decays, then its answer to k_t is replaced by a share
 * beta_t of v_t.  Shapes are those of mamba2_shape (b = batch, L = seqlen,
 * nh = nheads, H = headdim, S = dstate, G = ngroups; chunk_size is not used,
 * any valid value):
 *
 *   q, k         [b, L, G, S]   dtype   head h reads group h / (nh / G)
 *   v, y         [b, L, nh, H]  dtype
 *   g            [b, L, nh]     fp32    log decay, <= 0 (not checked)
 *   beta         [b, L, nh]     fp32    already activated, normally in [0, 1]
 *   initial_state, final_state [b, nh, S, H] fp32
 *   lengths      [b]            int32, NULL means L for every row
 *
 * With lengths, row b has min(max(lengths[b], 0), L) tokens: y is 0 past
 * them, final_state is the state after them, and nothing there is read into a
 * result (it may hold anything, NaN included). */
enum {
    /* q and k rows are divided by sqrt(sum of squares + l2_eps) (fp32). */
    MAMBA2_GDR_QK_L2NORM = 1
};

typedef struct {
    int64_t q_stride; /* elements from one token's q to the next (0: G * S); a  */
    int64_t k_stride; /* batch row is L of them.  Strides are at least the      */
    int64_t v_stride; /* row's own width.                        (v, 0: nh * H) */
    float scale;      /* factor of y, e.g. 1 / sqrt(S) */
    float l2_eps;     /* > 0 with MAMBA2_GDR_QK_L2NORM */
    int32_t flags;
    int32_t reserved; /* must be 0 */
} mamba2_gdr_options;

/* As for mamba2_ssd.h's calls: S and H up to 256, batch and nheads up to 65535,
 * else MAMBA2_ERR_UNSUPPORTED; so are tensors of more than 2^40 elements, strides
 * included.
 *
 * Whole sequences.  initial_state NULL means zeros; final_state NULL means not
 * written.  No workspace.  State arithmetic is fp32 on both dtypes: with bf16
 * inputs of S and H up to 128, both multiples of 8, and q, k, v whose address
 * and token stride are multiples of 16 bytes, the products run in chunks on the
 * tensor cores (but for a few tokens of few heads): what is added to the fp32 state is made of three bf16 parts
 * (24 bits) of every intermediate, from two parts (16 bits) of the state before
 * it; y takes two parts (16 bits) of the corrections and of the state.
 * Everything else runs token by token in fp32.  What is not finite: a NaN or an
 * infinity in a token's k, v or beta, or a NaN in its g, shows in its head's y from
 * that token on and in its final state; in chunks also, as NaN, in y of up to 15
 * tokens before it (those of its 16, counted from the sequence's start), since a
 * zero weight on a later token is a factor there.  In q it stays in its token. */
MAMBA2_API mamba2_status mamba2_gdr_fwd(const mamba2_shape* shape, const mamba2_gdr_options* options, const void* q,
                                        const void* k, const void* v, const float* g, const float* beta,
                                        const int32_t* lengths, const float* initial_state, void* y,
                                        float* final_state, struct CUstream_st* stream);

/* One token (shape->seqlen must be 1, else MAMBA2_ERR_INVALID_ARG): layouts
 * are mamba2_gdr_fwd's with L = 1, strides go from one batch row to the next.
 * state_in NULL means zeros; state_out is required and may be the same pointer
 * as state_in (update in place). */
MAMBA2_API mamba2_status mamba2_gdr_step(const mamba2_shape* shape, const mamba2_gdr_options* options, const void* q,
                                         const void* k, const void* v, const float* g, const float* beta,
                                         const float* state_in, float* state_out, void* y,
                                         struct CUstream_st* stream);

/* ------------------------------------------------------ causal convolution
 * Depthwise over time, channels last, W = width in 2 .. 8:
 *
 *     y_t = act(bias + sum_{w < W} weight[c, w] x_{t - (W - 1) + w}),
 *
 * act = SiLU with MAMBA2_CONV_SILU, else none; sums in fp32.
 *
 *   x, y         [b, L, C]      dtype
 *   weight       [C, W]         fp32    the last tap meets the current token
 *   bias         [C]            fp32, NULL means 0
 *   initial_state, final_state [b, W - 1, C] dtype: the W - 1 inputs before
 *                the first token, and the last W - 1 inputs, oldest first
 *                (initial_state NULL means zeros, final_state NULL not written)
 *   lengths      [b]            int32, as above
 * At most 65535 batch rows, 2^30 tokens and 2^30 channels. */
enum { MAMBA2_CONV_SILU = 1 };

typedef struct {
    int64_t batch, seqlen, channels, width;
    int64_t x_stride, y_stride; /* elements from token to token (0: channels) */
    int32_t dtype;              /* mamba2_dtype */
    int32_t flags;
} mamba2_conv_shape;

MAMBA2_API mamba2_status mamba2_causal_conv_fwd(const mamba2_conv_shape* shape, const void* x, const float* weight,
                                                const float* bias, const int32_t* lengths,
                                                const void* initial_state, void* y, void* final_state,
                                                struct CUstream_st* stream);

/* One token (shape->seqlen must be 1): state_in NULL means zeros; state_out is
 * required and may be the same pointer as state_in. */
MAMBA2_API mamba2_status mamba2_causal_conv_step(const mamba2_conv_shape* shape, const void* x, const float* weight,
                                                 const float* bias, const void* state_in, void* state_out, void* y,
                                                 struct CUstream_st* stream);

/* ------------------------------------------------------------- group norm
 * Per row (token) and group of channels / ngroups neighbouring channels:
 *
 *     u = x, or x SiLU(z) with MAMBA2_NORM_GATE_BEFORE
 *     u = u - mean(u)                      with MAMBA2_NORM_SUBTRACT_MEAN
 *     y = weight u / sqrt(mean(u^2) + eps) + bias
 *     y = y SiLU(z) with MAMBA2_NORM_GATE_AFTER, SiLU(y) with MAMBA2_NORM_SILU
 *
 * At most one of GATE_BEFORE, GATE_AFTER and SILU.  Statistics in fp32.
 *   x, z, y  [rows, channels] dtype; z only with a gate, else NULL
 *   weight, bias [channels] fp32; NULL means 1 and 0
 * channels % ngroups == 0, at most 32768 channels to a group, rows x ngroups below
 * 2^31 and rows x channels up to 2^40. */
enum {
    MAMBA2_NORM_SUBTRACT_MEAN = 1,
    MAMBA2_NORM_GATE_BEFORE = 2,
    MAMBA2_NORM_GATE_AFTER = 4,
    MAMBA2_NORM_SILU = 8
};

typedef struct {
    int64_t rows, channels, ngroups;
    int64_t x_stride, z_stride, y_stride; /* elements from row to row (0: channels) */
    float eps;                            /* > 0 */
    int32_t dtype;                        /* mamba2_dtype */
    int32_t flags;
    int32_t reserved; /* must be 0 */
} mamba2_norm_shape;

MAMBA2_API mamba2_status mamba2_group_norm(const mamba2_norm_shape* shape, const void* x, const void* z,
                                           const float* weight, const float* bias, void* y,
                                           struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA2_GATED_DELTA_H */
