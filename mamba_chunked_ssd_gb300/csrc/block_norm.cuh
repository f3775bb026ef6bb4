// block_norm.cuh — what the block norm's forward and backward kernels share: how rows come
// to the threads that keep them, and sums over a row whose channels lie with a block's
// threads or with those of a cluster's blocks.
#pragma once

#include "glr_math.cuh"

namespace m2 {
namespace bnorm {

using glr::add2;
using glr::f2;
using glr::fma2;
using glr::mul2;
using glr::sigmoid2;

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
// `most`: threads of a block, and of an SM at once.  Rows of one block where it has places for them; else, as long as eight
// take a row, blocks of half as many threads: while one waits for its cluster the SM has another.  In bf16, gated, backward
// 4096 x 8192 141 us, with blocks of 512 threads 153, 2048 x 8200 101 and 119; forward 2048 x 8200 52, with blocks of
// 1024 threads 65, 2048 x 16384 79 and 83; but backward 16384 x 4096 one block of 512 threads 187, two of 256 251.
inline Plan plan_of(int64_t rows, int64_t channels, int most) {
    Plan p = {1, 32, 1};
    const int resident = most;
    if (channels > most * kPer && channels <= 8 * (most / 2) * kPer) most /= 2;
    while (p.Q * (int64_t)most * kPer < channels) ++p.Q;
    p.threads = (int)((share_of(channels, p.Q) / kPer + 31) / 32 * 32);
    const int sms = sm_count();
    int64_t per_sm = resident / p.threads;
    per_sm = per_sm < 1 ? 1 : per_sm > 32 ? 32 : per_sm;
    const int64_t fit = per_sm * (int64_t)(sms > 0 ? sms : 152) / p.Q;
    p.walkers = imin64(rows, fit < 1 ? 1 : fit);
    return p;
}
// (`p.walkers` may become less.)
template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, int), const Args& a, Plan& p, int64_t rows, int bytes, cudaStream_t st) {
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.Q);
    cfg.blockDim = dim3((unsigned)p.threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.Q;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.Q > 1 ? 1 : 0;
    int there = 0;  // clusters that find places: they do not reach across the GPU's parts, which have odd numbers of SMs
    if (p.Q > 2 && p.walkers < rows) {
        if (cudaOccupancyMaxActiveClusters(&there, kernel, &cfg) == cudaSuccess && there > 0)
            p.walkers = imin64(p.walkers, there);
        else cudaGetLastError();
    }
    cfg.gridDim = dim3((unsigned)(p.walkers * p.Q));
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, kernel, a, p.Q);
    return launched == cudaSuccess ? cudaGetLastError() : (cudaGetLastError(), launched);
}

// Places for partial sums; two of each in turn, so that one barrier a sum is enough: who writes or sends to a place
// has met, since it was read, at the barrier (and the messages) of the sum between.
template <int N>
struct Sums {
    float warp[2][N][32];
    float block[2][8][N];
    glr::Mail mail;
};

// The blocks that share a row, and this one's place among them.
template <bool CLUSTER>
struct Share {
    int blocks, rank;
    unsigned int* status;
    __device__ __forceinline__ int Q() const { return CLUSTER ? blocks : 1; }
};

// The sum over a cluster's blocks of values that all threads of a block have; `count`: how many came before.
template <int N>
__device__ __forceinline__ void cluster_sums(float (&v)[N], Sums<N>& s, int count, const Share<true>& by) {
    float(*part)[N] = s.block[count & 1];
    if (threadIdx.x < by.Q()) {
#pragma unroll
        for (int k = 0; k < N; ++k) glr::send(&part[by.rank][k], &s.mail.bars[count & 1], threadIdx.x, v[k]);
    }
    glr::take_mail(s.mail, count, by.Q() * N * (int)sizeof(float), by.status);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = 0.f;
        for (int q = 0; q < by.Q(); ++q) v[k] += part[q][k];
    }
}

// A value's sum over a block's threads and over the Q blocks of a cluster, in a fixed order.
template <bool CLUSTER>
__device__ __forceinline__ void group_sums(float (&v)[1], Sums<1>& s, int& count, const Share<CLUSTER>& by) {
    float x = v[0];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    const int warps = blockDim.x / 32, lane = threadIdx.x & 31;
    if (warps > 1 || CLUSTER) {
        const int turn = count & 1;
        if (lane == 0) s.warp[turn][0][threadIdx.x >> 5] = x;
        __syncthreads();
        x = lane < warps ? s.warp[turn][0][lane] : 0.f;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    }
    v[0] = x;
    if constexpr (CLUSTER) cluster_sums(v, s, count, by);
    ++count;
}
// Three at once (and a fourth that is 0): half of the lanes go on with two of them, a quarter with each.
// Blocks of up to 16 warps.
template <bool CLUSTER>
__device__ __forceinline__ void group_sums(float (&v)[3], Sums<3>& s, int& count, const Share<CLUSTER>& by) {
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    const bool high = lane & 16, odd = lane & 8;
    float a = (high ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, high ? v[0] : v[2], 16);
    const float b = (high ? 0.f : v[1]) + __shfl_xor_sync(0xffffffffu, high ? v[1] : 0.f, 16);
    a = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);  // lanes 8 k .. 8 k + 7: value k
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
    if (warps > 1 || CLUSTER) {
        const int turn = count & 1;
        const int k = lane >> 3, w = lane & 7;
        if (w == 0 && k < 3) s.warp[turn][k][threadIdx.x >> 5] = a;
        __syncthreads();
        const float* from = s.warp[turn][k < 3 ? k : 2];
        a = (w < warps ? from[w] : 0.f) + (w + 8 < warps ? from[w + 8] : 0.f);
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] = __shfl_sync(0xffffffffu, a, 8 * k);
    if constexpr (CLUSTER) cluster_sums(v, s, count, by);
    ++count;
}

// How a thread's eight channels lie: in groups of GRP neighbouring ones, group i the (threadIdx + i blockDim)-th
// of the block's.  GRP > 1: rows start on a group's bytes and have whole groups, and a thread copies what it
// reads itself.  GRP = 1: rows lie in shared memory as they do in memory, from the 16-byte boundary
// before their start; the threads' copies are there for all after a barrier.  (In bf16, gated, backward: 16384 x 2050 in
// groups of two 228 us, 16384 x 2051 as whole rows 323.)
template <int GRP>
__device__ __forceinline__ int channel(int i) {
    return GRP * ((int)threadIdx.x + i / GRP * (int)blockDim.x) + i % GRP;
}

template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// 16 bytes, of which `bytes` are read and the others are zero.
__device__ __forceinline__ void copy_piece(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// A gate z as it comes, but no lower than -1000: SiLU is 0 from there down, and the product of z with what it gates stays
// a number at the dtype's lowest value, too.  NaN stays.  (As p (z sigmoid(z)) instead, which keeps z for longer,
// 8192 x 8192 in bf16 with an fp32 residual takes 185 us for 139, in registers that are all taken.)
__device__ __forceinline__ float gate(float z) { return glr::max_nan(z, -1000.f); }
__device__ __forceinline__ float2 gate(float2 z) { return make_float2(gate(z.x), gate(z.y)); }
__device__ __forceinline__ uint32_t gate(uint32_t z) {  // two of bf16
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(z), "r"(0xc47ac47au));
    return r;
}

// A walker's rows of one input.
template <typename E, int GRP>
struct RowIn {
    static constexpr int kGroups = kPer / GRP, kBytes = GRP * (int)sizeof(E);
    static constexpr bool kOwn = GRP > 1;
    using Unit = typename Word<kBytes>::type;
    const E* next;  // kOwn: this thread's first channel of the row that is fetched next; else the block's first
    bool first;  // (bf16, not kOwn) the row that is fetched next is less than 16 bytes behind the tensor's start

    static __host__ __device__ __forceinline__ int place_bytes(int threads) {
        return threads * kPer * (int)sizeof(E) + (kOwn ? 0 : 32);
    }
    __device__ __forceinline__ void start(const void* base, int64_t row, int64_t stride, int64_t c0) {
        next = static_cast<const E*>(base) + row * stride + c0 + (kOwn ? GRP * (int)threadIdx.x : 0);
        first = (row * stride + c0) * (int64_t)sizeof(E) < 16;
    }
    // zeros in the places of channels that are not there, which are never written again
    static __device__ __forceinline__ void clear(uint8_t* place, int n) {
        if constexpr (kOwn) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (channel<GRP>(i * GRP) >= n)
                    *reinterpret_cast<Unit*>(place + (i * blockDim.x + threadIdx.x) * kBytes) = {};
        }
    }
    __device__ __forceinline__ void fetch(uint8_t* place, int n, int64_t step) {
        const int tid = threadIdx.x;
        if constexpr (kOwn) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (channel<GRP>(i * GRP) < n)
                    copy_async<kBytes>(tc::smem_u32(place + (i * blockDim.x + tid) * kBytes), next + i * GRP * (int)blockDim.x);
        } else if constexpr (sizeof(E) == 4) {
            // the row's first elements up to the boundary, whole pieces of 16 bytes, the last elements
            constexpr int per = 4;
            const int skip = (int)(reinterpret_cast<uintptr_t>(next) & 15);
            const int head = min(((16 - skip) & 15) / 4, n), whole = (n - head) / per, tail = head + whole * per;
            const uint32_t to = tc::smem_u32(place + skip);
            for (int k = tid; k < whole; k += blockDim.x) copy_async<16>(to + 4 * (head + k * per), next + head + k * per);
            const int end = tid < per ? tid : tail + tid - per;  // this thread's element at an end
            if (tid < per ? tid < head : tid < 2 * per && end < n) copy_async<4>(to + 4 * end, next + end);
        } else {
            // Single elements are too small for an asynchronous copy: pieces of 16 bytes, of which the first begins up to 14
            // bytes before the row (in the tensor, or between its rows), and the last is read as far as the row goes.  Where
            // the first would begin before the tensor, its elements are stored.  (16384 x 2051 in bf16, gated, forward /
            // backward: 128 / 323 us, with a load and a store for each element of a row's ends 181 / 419.)
            const int from = (int)(reinterpret_cast<uintptr_t>(next) & 15), to = from + n * (int)sizeof(E);
            const uint8_t* at = reinterpret_cast<const uint8_t*>(next) - from;
            const bool single = first && from;
            for (int k = single ? tid + 1 : tid; k < to / 16; k += blockDim.x)
                copy_async<16>(tc::smem_u32(place + 16 * k), at + 16 * k);
            if (tid == 0 && to % 16 && !(single && to < 16))
                copy_piece(tc::smem_u32(place + to / 16 * 16), at + to / 16 * 16, to % 16);
            if (single && tid < min((16 - from) / (int)sizeof(E), n)) reinterpret_cast<E*>(place + from)[tid] = next[tid];
            first = false;
        }
        next += step;
    }
    // `row`: the row's first channel in memory (but kOwn); zeros where there is no channel.  GATE: values of a gate
    template <bool GATE = false>
    static __device__ __forceinline__ void read(const uint8_t* place, const E* row, int n, float2 (&f)[4]) {
        if constexpr (kOwn) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const Unit v = *reinterpret_cast<const Unit*>(place + (i * blockDim.x + threadIdx.x) * kBytes);
                const auto* p = reinterpret_cast<const typename glr::Pair<E>::raw*>(&v);
#pragma unroll
                for (int k = 0; k < GRP / 2; ++k) f[i * GRP / 2 + k] = glr::Pair<E>::get(GATE ? gate(p[k]) : p[k]);
            }
        } else {
            const E* from = reinterpret_cast<const E*>(place + (reinterpret_cast<uintptr_t>(row) & 15));
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = channel<GRP>(i);
                float v = c < n ? to_f32(from[c]) : 0.f;
                if (GATE) v = gate(v);
                if (i % 2) f[i / 2].y = v;
                else f[i / 2].x = v;
            }
        }
    }
};

// A walker's rows of one output.
template <typename E, int GRP>
struct RowOut {
    E* next;  // as RowIn's
    __device__ __forceinline__ void start(void* base, int64_t row, int64_t stride, int64_t c0) {
        next = static_cast<E*>(base) + row * stride + c0 + (GRP > 1 ? GRP * (int)threadIdx.x : 0);
    }
    __device__ __forceinline__ void write(int n, const float2 (&f)[4], int64_t step) {
        if constexpr (GRP > 1) {
#pragma unroll
            for (int i = 0; i < kPer / GRP; ++i) {
                typename Word<GRP * sizeof(E)>::type v;
                auto* p = reinterpret_cast<typename glr::Pair<E>::raw*>(&v);
#pragma unroll
                for (int k = 0; k < GRP / 2; ++k) p[k] = glr::Pair<E>::put(f[i * GRP / 2 + k]);
                if (channel<GRP>(i * GRP) < n) *reinterpret_cast<decltype(v)*>(next + i * GRP * (int)blockDim.x) = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = channel<GRP>(i);
                if (c < n) next[c] = from_f32<E>(i % 2 ? f[i / 2].y : f[i / 2].x);
            }
        }
        next += step;
    }
};

// A thread's values of a row of fp32 weights (`none` without one), and its sums to such a row.
template <int GRP>
__device__ __forceinline__ void load_weight(const float* w, int n, float none, float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = channel<GRP>(i);
        const float v = w && c < n ? w[c] : none;
        if (i % 2) f[i / 2].y = v;
        else f[i / 2].x = v;
    }
}
template <int GRP>
__device__ __forceinline__ void store_weight(float* w, int n, const float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = channel<GRP>(i);
        if (c < n) w[c] = i % 2 ? f[i / 2].y : f[i / 2].x;
    }
}

__device__ __forceinline__ float sum_of(const float2& v) { return v.x + v.y; }

// The widest groups that a call's rows allow: `t` and `r`, all addresses and strides in bytes of the two dtypes' tensors
// or-ed together.  Eight channels only where both are bf16 (16 bytes of fp32 are four).
inline int group_of(uint64_t t, uint64_t r, int64_t channels, int t_bytes, int r_bytes) {
    for (int g = t_bytes == 2 && r_bytes == 2 ? 8 : 4; g > 1; g /= 2)
        if (channels % g == 0 && t % (uint64_t)(g * t_bytes) == 0 && r % (uint64_t)(g * r_bytes) == 0) return g;
    return 1;
}

}  // namespace bnorm
}  // namespace m2
