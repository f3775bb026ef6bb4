// glr_math.cuh — the gated linear recurrence's arithmetic for two channels at
// once (packed fp32 operations), and the parts that its forward and backward
// kernels share: where a warp's tokens lie in shared memory and how they come there.
#pragma once

#include "gated_linear.cuh"
#include "tc_ptx.cuh"

namespace m2 {
namespace glr {

using namespace tc;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 8;                  // tokens of a warp
constexpr int kTile = kWarps * kTok;     // tokens of a block's step
constexpr int kStrip = 64;               // channels of a block: two to a lane
static_assert(kTile == MAMBA2_GLR_CHUNK, "a chunk state is the state that enters a tile");

__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The larger of the two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 1 / (1 + e^-x) by the hardware's exponential and reciprocal, for both dtypes: a few 1e-7 of
// it for |x| of the gates' size (the exponent's rounding to fp32, 2^-24 |x| log2 e, leads), no
// error that grows along the sequence, since log a takes it as a relative error.  0 at -infinity, 1 at infinity.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 t = mul2(x, f2(-kLog2e));
    const float2 d = add2(f2(1.f), make_float2(ex2_approx(t.x), ex2_approx(t.y)));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// a = e^la and m = 1 - a^2 of la <= 0.  With la = n ln 2 + y, |y| <= ln 2 / 2, the Taylor
// polynomial p of e^y - 1 to y^7 (remainder 2e-8 of p) gives e^la - 1 = 2^n p + (2^n - 1)
// without cancellation, so that m keeps its precision for a next to 1, where it sets the
// state's scale, and a is e^la rounded: an error of a that is the same for every token would be
// multiplied by the recurrence's memory 1 / (1 - a).  Below -87 a is 1.6e-38.
__device__ __forceinline__ void decay2(float2 la, float2& a, float2& m) {
    la.x = max_nan(la.x, -87.f), la.y = max_nan(la.y, -87.f);
    const float2 big = f2(12582912.f);  // 1.5 2^23: its sum with a small number is rounded to a whole one
    const float2 t = fma2(la, f2(kLog2e), big);
    const float2 y = fma2(add2(t, f2(-12582912.f)), f2(-0.693147180559945f), la);
    float2 p = fma2(y, f2(1.f / 5040.f), f2(1.f / 720.f));
    p = fma2(p, y, f2(1.f / 120.f));
    p = fma2(p, y, f2(1.f / 24.f));
    p = fma2(p, y, f2(1.f / 6.f));
    p = fma2(p, y, f2(0.5f));
    p = fma2(p, y, f2(1.f));
    p = mul2(p, y);
    // 2^n from the bits that hold n
    const float2 s = make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                                 __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u));
    a = fma2(s, p, s);
    const float2 e = fma2(s, p, add2(s, f2(-1.f)));  // a - 1
    m = mul2(e, fma2(e, f2(-1.f), f2(-2.f)));        // -e (e + 2)
}

// 1 / sqrt(m), finite at m = 0 (where log a, which it meets, is 0 too).
__device__ __forceinline__ float2 rsqrt2(float2 m) {
    return make_float2(rsqrt_approx(fmaxf(m.x, 1e-36f)), rsqrt_approx(fmaxf(m.y, 1e-36f)));
}

// A pair of neighbouring channels as it lies in memory.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using raw = uint32_t;
    static __device__ __forceinline__ float2 get(raw v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ raw put(float2 v) { return pack_bf16x2(v.x, v.y); }
};
template <>
struct Pair<float> {
    using raw = float2;
    static __device__ __forceinline__ float2 get(raw v) { return v; }
    static __device__ __forceinline__ raw put(float2 v) { return v; }
};

// How rows lie: on 16 bytes with whole 16-byte pieces of channels, on a pair of channels, or on an element.
enum Rows { kRows16, kRowsPair, kRowsOne };

// One sequence tensor of a block: its strip of channels, its batch row.
template <typename T>
struct Seq {
    const T* p;  // channel 0 of the strip, token 0
    int64_t stride;
};

// The tokens t .. t + 7 (those before n) of a strip with `have` channels into a warp's place in
// shared memory, [8][64] T; what is not there becomes 0.  A warp's lanes fill the place
// together: cp.async (waited for with its group, then __syncwarp), or plain loads where rows
// start on single bf16 elements.
template <typename T, Rows ROWS>
__device__ __forceinline__ void fetch(T* place, const Seq<T>& s, int64_t t, int64_t n, int have, int lane) {
    if constexpr (ROWS == kRows16) {
        constexpr int per = 16 / sizeof(T), across = kStrip / per, at_once = 32 / across;
        const int c = lane % across * per;
#pragma unroll
        for (int k = 0; k < kTok / at_once; ++k) {
            const int row = lane / across + k * at_once;
            const bool live = t + row < n && c < have;
            const T* from = live ? s.p + (t + row) * s.stride + c : s.p;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place + row * kStrip + c)),
                         "l"(from), "r"(live ? 16 : 0)
                         : "memory");
        }
    } else if constexpr (ROWS == kRowsPair) {
        constexpr int bytes = 2 * sizeof(T);
#pragma unroll
        for (int row = 0; row < kTok; ++row) {
            const bool live = t + row < n && 2 * lane < have;
            const T* from = live ? s.p + (t + row) * s.stride + 2 * lane : s.p;
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                             smem_u32(place + row * kStrip + 2 * lane)),
                         "l"(from), "n"(bytes), "r"(live ? bytes : 0)
                         : "memory");
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int row = 0; row < kTok; ++row)
#pragma unroll
            for (int c = lane; c < kStrip; c += 32) {
                const bool live = t + row < n && c < have;
                const T* from = live ? s.p + (t + row) * s.stride + c : s.p;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(place + row * kStrip + c)),
                             "l"(from), "r"(live ? 4 : 0)
                             : "memory");
            }
    } else {
        T v[kTok][2];
#pragma unroll
        for (int row = 0; row < kTok; ++row)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = lane + 32 * k;
                v[row][k] = t + row < n && c < have ? s.p[(t + row) * s.stride + c] : from_f32<T>(0.f);
            }
#pragma unroll
        for (int row = 0; row < kTok; ++row)
#pragma unroll
            for (int k = 0; k < 2; ++k) place[row * kStrip + lane + 32 * k] = v[row][k];
    }
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_for() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A pair of channels of a row to memory; `have` of the strip's channels are there.
template <typename T, bool ODD>
__device__ __forceinline__ void store(T* row, float2 v, int lane, int have) {
    if constexpr (!ODD) {
        if (2 * lane < have) *reinterpret_cast<typename Pair<T>::raw*>(row + 2 * lane) = Pair<T>::put(v);
    } else {
        if (2 * lane < have) row[2 * lane] = from_f32<T>(v.x);
        if (2 * lane + 1 < have) row[2 * lane + 1] = from_f32<T>(v.y);
    }
}

// fp32 values of a pair of channels, of which `have` of the strip's are there.
__device__ __forceinline__ float2 load_pair(const float* p, int lane, int have) {
    return make_float2(2 * lane < have ? p[2 * lane] : 0.f, 2 * lane + 1 < have ? p[2 * lane + 1] : 0.f);
}

// Blocks of a cluster split a sequence: each takes every K-th tile, and they exchange their tiles' summaries.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const void* here, uint32_t rank, float4 v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(here)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// How all of a call's rows lie (pointers that are null do not count).
inline Rows rows_of(const void* const* p, const int64_t* strides, int count, int64_t channels, int bytes) {
    uint64_t all = (uint64_t)channels * bytes;
    for (int k = 0; k < count; ++k) all |= reinterpret_cast<uintptr_t>(p[k]) | (uint64_t)strides[k] * bytes;
    return all % 16 == 0 ? kRows16 : all % (2 * bytes) == 0 ? kRowsPair : kRowsOne;
}

// Blocks that split a sequence: doubled up to 8, while there are fewer than four to an SM and tiles for them.
inline int glr_cluster(int64_t strips, int64_t tiles) {
    const int sms = sm_count();
    int K = 1;
    while (K < 8 && 2 * K <= tiles && strips * K < 4 * (int64_t)(sms > 0 ? sms : 152)) K *= 2;
    return K;
}

// A block for each strip of each batch row, or K of them as a cluster.
template <typename Args>
cudaError_t launch_strips(void (*kernel)(Args, int), const Args& a, int64_t strips, int K, int bytes, cudaStream_t st) {
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(strips * K), (unsigned)a.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)K;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = K > 1 ? 1 : 0;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, kernel, a, K);
    return launched == cudaSuccess ? cudaGetLastError() : (cudaGetLastError(), launched);
}

}  // namespace glr
}  // namespace m2
