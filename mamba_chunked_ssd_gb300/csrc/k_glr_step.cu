// k_glr_step.cu — one token of the gated linear recurrence for every batch row:
//
//   h = a h + sqrt(1 - a^2) sigmoid(i) x,  log a = A sigmoid(r),  y = h [SiLU(z)]
//
// A thread has two channels of one row.  The states (fp32) are most of the bytes.
#include "glr_math.cuh"

namespace m2 {
namespace {

using namespace glr;

constexpr int kBlock = 128;

template <typename T, bool ODD, bool GATED>
__global__ void __launch_bounds__(kBlock) k_glr_step(const GlrArgs a) {
    using P = Pair<T>;
    using Raw = typename P::raw;
    const int64_t c = ((int64_t)blockIdx.x * kBlock + threadIdx.x) * 2;
    if (c >= a.channels) return;
    const int have = (int)imin64(a.channels - c, 2);
    const int64_t b = blockIdx.y;
    auto pair = [&](const void* p, int64_t stride) {
        const T* q = static_cast<const T*>(p) + b * stride + c;
        if (!ODD) return P::get(*reinterpret_cast<const Raw*>(q));
        return make_float2(to_f32(q[0]), have > 1 ? to_f32(q[1]) : 0.f);
    };
    const float2 x = pair(a.x, a.x_stride), r = pair(a.r, a.r_stride), i = pair(a.i, a.i_stride);
    const float2 A = load_pair(a.A + c, 0, have);
    float2 h = a.init ? load_pair(a.init + b * a.channels + c, 0, have) : f2(0.f);
    float2 f, m;
    decay2<true>(mul2(A, sigmoid2(r)), f, m);
    h = fma2(f, h, mul2(mul2(sqrt2(m), sigmoid2(i)), x));
    store<float, true>(a.final_state + b * a.channels + c, h, 0, have);
    if (GATED) {
        const float2 z = pair(a.z, a.z_stride);
        h = mul2(h, mul2(z, sigmoid2(z)));
    }
    store<T, ODD>(static_cast<T*>(a.y) + b * a.y_stride + c, h, 0, have);
}

template <typename T>
cudaError_t launch_t(const GlrArgs& a, cudaStream_t st) {
    const void* p[] = {a.x, a.r, a.i, a.z, a.y};
    const int64_t strides[] = {a.x_stride, a.r_stride, a.i_stride, a.z ? a.z_stride : 0, a.y_stride};
    const bool odd = rows_of(p, strides, 5, a.channels, sizeof(T)) == kRowsOne;
    const dim3 grid((unsigned)((a.channels + 2 * kBlock - 1) / (2 * kBlock)), (unsigned)a.batch);
    if (odd) {
        if (a.z) k_glr_step<T, true, true><<<grid, kBlock, 0, st>>>(a);
        else k_glr_step<T, true, false><<<grid, kBlock, 0, st>>>(a);
    } else {
        if (a.z) k_glr_step<T, false, true><<<grid, kBlock, 0, st>>>(a);
        else k_glr_step<T, false, false><<<grid, kBlock, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glr_step(const GlrArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
