// gated_delta.cuh — arguments and launchers of the gated-delta-rule layer's
// kernels (the gated delta rule, the causal convolution, the group norm).
// Arguments were validated by the C-ABI layer; strides are resolved (never 0).
#pragma once

#include "common.cuh"

namespace m2 {

struct GdrArgs {
    Geom g;  // chunk is not used
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;  // elements from token to token
    const float* gate;                     // log decay
    const float* beta;
    const int32_t* lengths;  // may be null
    const float* init;       // may be null; the step: may equal final_state
    void* y;
    float* final_state;  // may be null (not in the step)
    float scale, l2_eps;
    bool l2norm;
};

struct ConvArgs {
    int64_t batch, seqlen, channels;
    int width;
    int64_t x_stride, y_stride;
    const void* x;
    const float* weight;
    const float* bias;       // may be null
    const int32_t* lengths;  // may be null
    const void* init;        // may be null; the step: may equal final_state
    void* y;
    void* final_state;  // may be null (not in the step)
    bool silu;
};

struct NormArgs {
    int64_t rows, channels, ngroups;
    int64_t x_stride, z_stride, y_stride;
    const void* x;
    const void* z;  // with a gate
    const float* weight;
    const float* bias;
    void* y;
    float eps;
    int flags;
};

// Tokens of batch row b: lengths[b] clamped to 0 .. L.
__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t L) {
    if (!lengths) return L;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n < L ? n : L);
}

// x / (1 + e^-x).  Values that leave as bf16 take the fast exponential and
// reciprocal (relative error about 1.5e-6 for |x| < 16: the exponent's rounding to fp32 is
// 1e-6 of it, exponential and reciprocal the rest; bf16's is 2e-3; from x = -127 ln 2 on
// the quotient is 0, its limit).
__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <typename T>
__device__ __forceinline__ float silu_f32(float x) {
    if (sizeof(T) == 2) return x * rcp_approx(1.f + ex2_approx(-kLog2e * x));
    return x / (1.f + expf(-x));
}

// N consecutive elements as fp32, N * sizeof(T) <= 16 bytes, one load of that
// size (the pointer aligned to it), and back.
template <typename T, int N>
struct VecOf;
template <>
struct VecOf<float, 4> { using type = float4; };
template <>
struct VecOf<float, 2> { using type = float2; };
template <>
struct VecOf<float, 1> { using type = float; };
template <>
struct VecOf<__nv_bfloat16, 8> { using type = uint4; };
template <>
struct VecOf<__nv_bfloat16, 4> { using type = uint2; };
template <>
struct VecOf<__nv_bfloat16, 2> { using type = uint32_t; };
template <>
struct VecOf<__nv_bfloat16, 1> { using type = __nv_bfloat16; };

template <int N>
__device__ __forceinline__ void unpack(const typename VecOf<float, N>::type& r, float (&f)[N], const float*) {
    const float* p = reinterpret_cast<const float*>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = p[i];
}
template <int N>
__device__ __forceinline__ void unpack(const typename VecOf<__nv_bfloat16, N>::type& r, float (&f)[N],
                                       const __nv_bfloat16*) {
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __bfloat162float(p[i]);
}
template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::type pack(const float (&f)[N]) {
    typename VecOf<T, N>::type r;
    T* p = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = from_f32<T>(f[i]);
    return r;
}

cudaError_t launch_gdr_fwd(const GdrArgs& a, bool bf16, cudaStream_t st);
// The chunked kernel on the tensor cores (bf16) and the calls it covers.
bool gdr_chunk_tc_fits(const GdrArgs& a);
cudaError_t launch_gdr_chunk_tc(const GdrArgs& a, cudaStream_t st);
cudaError_t launch_gdr_recurrent(const GdrArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_gdr_step(const GdrArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_causal_conv(const ConvArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_causal_conv_step(const ConvArgs& a, bool bf16, cudaStream_t st);
cudaError_t launch_group_norm(const NormArgs& a, bool bf16, cudaStream_t st);

}  // namespace m2
