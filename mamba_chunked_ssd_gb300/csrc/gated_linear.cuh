// gated_linear.cuh — arguments and launchers of the recurrent block's kernels
// (gated linear recurrence, block norm, gradient of the causal convolution).
// Arguments were validated by the C-ABI layer; strides are resolved (never 0).
#pragma once

#include "gated_delta.cuh"
#include "mamba2_gated_linear.h"

namespace m2 {

struct GlrArgs {
    int64_t batch, seqlen, channels;
    int64_t x_stride, r_stride, i_stride, z_stride, y_stride;  // elements from token to token
    const void* x;
    const void* r;
    const void* i;
    const void* z;  // may be null
    const float* A;
    const int32_t* lengths;  // may be null
    const float* init;       // may be null; the step: may equal final_state
    void* y;
    float* chunk_states;  // may be null
    float* final_state;   // may be null (not in the step)
    unsigned int* status = nullptr;  // the device's status word, for clusters
    int64_t first;        // strip of channels (of all batch rows) that clusters start with, and single blocks end before
};

struct GlrBwdArgs {
    int64_t batch, seqlen, channels;
    int64_t x_stride, r_stride, i_stride, z_stride, dy_stride;
    int64_t dx_stride, dr_stride, di_stride, dz_stride;
    const void* dy;
    const void* x;
    const void* r;
    const void* i;
    const void* z;  // may be null, dz with it
    const float* A;
    const int32_t* lengths;  // may be null
    const float* chunk_states;
    const float* dfinal;  // may be null
    void* dx;
    void* dr;
    void* di;
    void* dz;
    float* dA;
    float* dinit;     // may be null
    float* partials;    // [batch, channels]: each row's part of A dA
    int64_t first;    // as GlrArgs'
};

struct ConvBwdArgs {
    int64_t batch, seqlen, channels;
    int width;
    int64_t x_stride, dy_stride, dx_stride;
    const void* dy;
    const void* x;
    const float* weight;
    const float* bias;       // may be null
    const int32_t* lengths;  // may be null
    const void* init;        // may be null
    const void* dfinal;      // may be null
    void* dx;
    float* dweight;
    float* dbias;  // may be null
    void* dinit;   // may be null
    bool silu;
    float* partials;
};

struct BlockNormArgs {
    int64_t rows, channels;
    int64_t x_stride, z_stride, res_stride, out_stride, y_stride;
    const void* x;
    const void* z;    // may be null
    const void* res;  // may be null; may equal out
    const float* post_weight;  // weights may be null: 1
    const float* scale;
    const float* pre_weight;
    void* out;
    void* y;  // with the norm before
    float eps;
    bool post, pre;
    unsigned int* status = nullptr;  // the device's status word, for clusters
};

struct BlockNormBwdArgs {
    int64_t rows, channels;
    int64_t x_stride, z_stride, out_stride, dy_stride;
    int64_t dx_stride, dz_stride, dout_stride, dres_stride;
    const void* dout;  // may be null
    const void* dy;    // with the norm before
    const void* x;
    const void* z;    // may be null, dz with it
    const void* out;  // with the norm before
    const float* post_weight;
    const float* scale;
    const float* pre_weight;
    void* dx;
    void* dz;
    void* dres;  // may be null; may equal dout
    float* dpost;  // may be null
    float* dscale;
    float* dpre;
    float eps;
    bool post, pre;
    float* partials;
    unsigned int* status = nullptr;  // the device's status word, for clusters
};

// out[c] = sum over k < rows of partials[k, c] (/ by[c]), for up to three outputs that lie side by
// side in a row of partials; one that is null is left out.  The sums' order depends on
// `rows` alone.
struct SumOut {
    float* out;
    int64_t len;
};
cudaError_t launch_sum_rows(const float* partials, int64_t rows, SumOut o0, SumOut o1, SumOut o2, const float* by,
                            cudaStream_t st);

cudaError_t launch_glr_fwd(const GlrArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_glr_step(const GlrArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_glr_bwd(const GlrBwdArgs& a, bool bf16, cudaStream_t st);

// Floats of dweight's and dbias's parts.
int64_t conv_bwd_partials(int64_t batch, int64_t seqlen, int64_t channels, int width);
cudaError_t launch_causal_conv_bwd(const ConvBwdArgs& a, bool bf16, cudaStream_t st);

cudaError_t launch_block_norm(const BlockNormArgs& a, bool bf16, bool res_bf16, cudaStream_t st);
// Floats of the weights' gradients' parts.
int64_t block_norm_bwd_partials(int64_t rows, int64_t channels);
cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool bf16, bool res_bf16, cudaStream_t st);

}  // namespace m2
