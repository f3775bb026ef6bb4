// k_group_norm.cu — group norm over each row's groups of channels, with a gate
// or an activation:
//
//   u = x [SiLU(z)];  u -= mean(u) [if asked];  y = w u / sqrt(mean(u^2) + eps) + bias;
//   y *= SiLU(z), or y = SiLU(y) [if asked]
//
// x (and z) are read once and y is written once: the kernel is bound by
// memory.  A group lives in the registers of TPG threads (a part of a warp, a
// warp, or a block), so the mean and then the squares of the differences from
// it are summed from registers, in fp32 and a fixed order, without a second
// read.
#include "gated_delta.cuh"
#include "mamba2_gated_delta.h"

namespace m2 {
namespace {

constexpr int kWarpBlock = 256;  // threads of a block whose groups stay inside warps

// Sum over the group's threads.
template <int TPG>
__device__ __forceinline__ float group_sum(float v, float* smem) {
#pragma unroll
    for (int m = (TPG < 32 ? TPG : 32) / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (TPG > 32) {
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
        __syncthreads();
        v = smem[threadIdx.x & 31 & (TPG / 32 - 1)];
#pragma unroll
        for (int m = TPG / 64; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    }
    return v;
}

// VEC elements per load, NV loads per thread, TPG threads per group.
template <typename T, int VEC, int NV, int TPG>
__global__ void __launch_bounds__(TPG > 32 ? TPG : kWarpBlock) k_group_norm(const NormArgs a) {
    using V = typename VecOf<T, VEC>::type;
    __shared__ float smem[32];
    const int lane = threadIdx.x % TPG;
    const int64_t per = TPG > 32 ? 1 : kWarpBlock / TPG;
    int64_t seg = (int64_t)blockIdx.x * per + threadIdx.x / TPG;
    const bool live = seg < a.rows * a.ngroups;
    if (!live) seg = 0;  // stays for the warp's shuffles
    const int64_t row = seg / a.ngroups, grp = seg - row * a.ngroups;
    const int size = (int)(a.channels / a.ngroups), nvec = size / VEC;
    const int64_t c0 = grp * size;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + c0;
    const bool before = (a.flags & MAMBA2_NORM_GATE_BEFORE) != 0, after = (a.flags & MAMBA2_NORM_GATE_AFTER) != 0;
    const bool gated = before || after;

    V xr[NV], zr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * TPG;
        xr[i] = V{};
        if (j < nvec) xr[i] = *reinterpret_cast<const V*>(x + (int64_t)j * VEC);
    }
    if (gated) {
        const T* z = static_cast<const T*>(a.z) + row * a.z_stride + c0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * TPG;
            zr[i] = V{};
            if (j < nvec) zr[i] = *reinterpret_cast<const V*>(z + (int64_t)j * VEC);
        }
    }
    float u[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        unpack<VEC>(xr[i], u[i], (const T*)nullptr);
        if (before) {
            float z[VEC];
            unpack<VEC>(zr[i], z, (const T*)nullptr);
#pragma unroll
            for (int e = 0; e < VEC; ++e) u[i][e] *= silu_f32<T>(z[e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += u[i][e];
    }
    float mean = 0.f;
    if (a.flags & MAMBA2_NORM_SUBTRACT_MEAN) mean = group_sum<TPG>(s, smem) / (float)size;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (lane + i * TPG < nvec) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                u[i][e] -= mean;
                ss = fmaf(u[i][e], u[i][e], ss);
            }
        }
    }
    const float r = rsqrtf(group_sum<TPG>(ss, smem) / (float)size + a.eps);
    if (!live) return;
    T* y = static_cast<T*>(a.y) + row * a.y_stride + c0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * TPG;
        if (j >= nvec) break;
        const int64_t c = c0 + (int64_t)j * VEC;
        float w[VEC], o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[e] = a.weight ? a.weight[c + e] : 1.f;
            o[e] = u[i][e] * r * w[e];
        }
        if (a.bias) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] += a.bias[c + e];
        }
        if (after) {
            float z[VEC];
            unpack<VEC>(zr[i], z, (const T*)nullptr);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] *= silu_f32<T>(z[e]);
        } else if (a.flags & MAMBA2_NORM_SILU) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = silu_f32<T>(o[e]);
        }
        *reinterpret_cast<V*>(y + (int64_t)j * VEC) = pack<T, VEC>(o);
    }
}

template <typename T, int VEC, int NV, int TPG>
cudaError_t launch_n(const NormArgs& a, cudaStream_t st) {
    const int64_t per = TPG > 32 ? 1 : kWarpBlock / TPG;
    const int64_t blocks = (a.rows * a.ngroups + per - 1) / per;
    k_group_norm<T, VEC, NV, TPG><<<(unsigned)blocks, TPG > 32 ? TPG : kWarpBlock, 0, st>>>(a);
    return cudaGetLastError();
}

// The fewest threads that hold the group.
template <typename T, int VEC>
cudaError_t launch_v(const NormArgs& a, cudaStream_t st) {
    const int64_t n = a.channels / a.ngroups / VEC;
    constexpr int K = VEC == 1 ? 8 : 1;  // single elements: more loads per thread
    if (n <= 8 * K) return launch_n<T, VEC, K, 8>(a, st);
    if (n <= 16 * K) return launch_n<T, VEC, K, 16>(a, st);
    if (n <= 32 * K) return launch_n<T, VEC, K, 32>(a, st);
    if (n <= 64 * K) return launch_n<T, VEC, 2 * K, 32>(a, st);
    if (n <= 128 * K) return launch_n<T, VEC, K, 128>(a, st);
    if (n <= 256 * K) return launch_n<T, VEC, 2 * K, 128>(a, st);
    if (n <= 512 * K) return launch_n<T, VEC, 2 * K, 256>(a, st);
    if (n <= 1024 * K) return launch_n<T, VEC, 2 * K, 512>(a, st);
    if (n <= 2048 * K) return launch_n<T, VEC, 2 * K, 1024>(a, st);
    if (n <= 4096 * K) return launch_n<T, VEC, 4 * K, 1024>(a, st);
    return launch_n<T, VEC, 8 * K, 1024>(a, st);
}

template <typename T>
cudaError_t launch_t(const NormArgs& a, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                        reinterpret_cast<uintptr_t>(a.z);
    const bool vec = (a.channels / a.ngroups) % VEC == 0 && a.x_stride % VEC == 0 && a.y_stride % VEC == 0 &&
                     a.z_stride % VEC == 0 && (p & 15) == 0;
    return vec ? launch_v<T, VEC>(a, st) : launch_v<T, 1>(a, st);
}

}  // namespace

cudaError_t launch_group_norm(const NormArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
