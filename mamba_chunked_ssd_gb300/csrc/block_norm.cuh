// block_norm.cuh — what the block norm's forward and backward kernels share: sums over a
// row whose channels lie with the threads of a warp, of a block or of a cluster's blocks,
// and rows on their way to the thread that reads them.
#pragma once

#include "glr_math.cuh"

namespace m2 {
namespace bnorm {

constexpr int kPer = 8;  // channels of a thread

// A block's channels of a row that Q blocks share: a multiple of eight, less in the last block.
__host__ __device__ __forceinline__ int64_t share_of(int64_t channels, int Q) {
    return ((channels + Q - 1) / Q + kPer - 1) / kPer * kPer;
}

// Blocks that share a row, threads of a block, and walkers down the rows.
struct Plan {
    int Q, threads;
    int64_t walkers;
};
// `resident`: threads of an SM at once.
inline Plan plan_of(int64_t rows, int64_t channels, int resident) {
    Plan p = {1, 32, 1};
    while (p.Q * 512 * kPer < channels) p.Q *= 2;
    while (p.threads < 512 && p.threads * kPer < channels) p.threads *= 2;
    const int sms = sm_count();
    int64_t per_sm = resident / p.threads;
    if (per_sm > 32) per_sm = 32;
    const int64_t fit = per_sm * (int64_t)(sms > 0 ? sms : 152) / p.Q;
    p.walkers = imin64(rows, fit < 1 ? 1 : fit);
    return p;
}
template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, int), const Args& a, const Plan& p, int threads, int bytes,
                        cudaStream_t st) {
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.walkers * p.Q));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.Q;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.Q > 1 ? 1 : 0;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, kernel, a, p.Q);
    return launched == cudaSuccess ? cudaGetLastError() : (cudaGetLastError(), launched);
}

// Places for partial sums; two of each in turn, so that one barrier a sum is enough: who
// writes a place has met, since it was read, at the barrier of the sum between.
template <int N>
struct Sums {
    float warp[2][32][N];
    float block[2][8][N];
};

// Sums of N values over TPG threads (a warp, or a block, which then is all of its threads)
// and over the Q blocks of a cluster, in a fixed order.
template <int TPG, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], Sums<N>& s, int& turn, int Q, int rank) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
    if constexpr (TPG > 32) {
        constexpr int warps = TPG / 32;
        turn ^= 1;
        const int lane = threadIdx.x & 31;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) s.warp[turn][threadIdx.x >> 5][k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = s.warp[turn][lane & (warps - 1)][k];
#pragma unroll
        for (int m = warps / 2; m > 0; m >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
        if (Q > 1) {
            if (threadIdx.x < Q) {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    uint32_t at;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                                 : "=r"(at)
                                 : "r"(tc::smem_u32(&s.block[turn][rank][k])), "r"(threadIdx.x));
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v[k]) : "memory");
                }
            }
            glr::cluster_sync();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                v[k] = 0.f;
                for (int q = 0; q < Q; ++q) v[k] += s.block[turn][q][k];
            }
        }
    }
}

// N elements that start on their own size (up to 16 bytes: their pieces' size) as fp32, and back.
template <typename R, int N>
struct Piece {
    static constexpr int kPer = 16 / sizeof(R) < N ? 16 / (int)sizeof(R) : N;
    typename VecOf<R, kPer>::type v[N / kPer];
};
template <typename R, int N>
__device__ __forceinline__ void load_piece(Piece<R, N>& p, const R* from) {
#pragma unroll
    for (int k = 0; k < N / Piece<R, N>::kPer; ++k)
        p.v[k] = reinterpret_cast<const typename VecOf<R, Piece<R, N>::kPer>::type*>(from)[k];
}
template <typename R, int N>
__device__ __forceinline__ void widen(const Piece<R, N>& p, float (&f)[N]) {
    constexpr int per = Piece<R, N>::kPer;
#pragma unroll
    for (int k = 0; k < N / per; ++k) {
        float g[per];
        unpack<per>(p.v[k], g, (const R*)nullptr);
#pragma unroll
        for (int e = 0; e < per; ++e) f[k * per + e] = g[e];
    }
}
template <typename R, int N>
__device__ __forceinline__ void store_piece(R* to, const float (&f)[N]) {
    constexpr int per = Piece<R, N>::kPer;
#pragma unroll
    for (int k = 0; k < N / per; ++k) {
        float g[per];
#pragma unroll
        for (int e = 0; e < per; ++e) g[e] = f[k * per + e];
        reinterpret_cast<typename VecOf<R, per>::type*>(to)[k] = pack<R, per>(g);
    }
}

// An aligned piece into shared memory, waited for with its group.
template <typename R, int N>
__device__ __forceinline__ void copy_piece(Piece<R, N>* to, const R* from) {
    constexpr int bytes = sizeof(Piece<R, N>) < 16 ? (int)sizeof(Piece<R, N>) : 16;
#pragma unroll
    for (int k = 0; k < (int)sizeof(Piece<R, N>) / bytes; ++k) {
        const uint32_t dst = tc::smem_u32(reinterpret_cast<uint8_t*>(to) + k * bytes);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(from) + k * bytes;
        if constexpr (bytes == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(bytes) : "memory");
    }
}

// sigmoid of a gate: the hardware's exponential and reciprocal for bf16, exact functions else.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if (sizeof(T) == 2) return rcp_approx(1.f + ex2_approx(-kLog2e * z));
    return 1.f / (1.f + expf(-z));
}

}  // namespace bnorm
}  // namespace m2
