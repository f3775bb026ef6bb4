// glr_math.cuh — the gated linear recurrence's arithmetic for two channels at
// once (packed fp32 operations), and the parts that its forward and backward
// kernels share: where a warp's tokens lie in shared memory and how they come there.
#pragma once

#include "gated_linear.cuh"
#include "tc_ptx.cuh"


namespace m2 {
namespace glr {

using namespace tc;

constexpr int kGroups = 8;               // groups of lanes in a block, each with its own tokens
constexpr int kTok = 8;                  // tokens of a group
constexpr int kTile = kGroups * kTok;    // tokens of a block's step
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

// a = e^la and m = 1 - a^2 of la <= 0.  A polynomial p of e^la - 1 keeps m's precision for a
// next to 1, where m sets the state's scale, and gives an a that is e^la rounded: an error of a that is the
// same for every token would be multiplied by the recurrence's memory 1 / (1 - a), and p's is a share of 1 - a.
// p / la to la^6 by a Remez exchange for the relative error on -1 .. 0 (9.3e-9 with these fp32 coefficients).  WIDE, where A
// is below -1:
// la = n ln 2 + y, |y| <= ln 2 / 2, and e^la - 1 = 2^n p + (2^n - 1) without cancellation, p / y
// to y^5 (3.1e-8); below -87 (kLeastLog) a is 1.6e-38.
// A strip takes the wide form for any A below -1 (forward, 16 x 2048 x 4096 in bf16: 177 us with the narrow one, 193 with
// the wide one; forward and backward, 4 x 4096 x 4096, gated: 137 and 252, 146 and 263).
constexpr float kLeastLog = -87.f;
template <bool WIDE>
__device__ __forceinline__ void decay2(float2 la, float2& a, float2& m) {
    float2 e;  // a - 1
    if constexpr (!WIDE) {
        e = fma2(la, f2(0.00012913094542454928f), f2(0.001301126554608345f));
        e = fma2(e, la, f2(0.008276209235191345f));
        e = fma2(e, la, f2(0.04164746776223183f));
        e = fma2(e, la, f2(0.16666366159915924f));
        e = fma2(e, la, f2(0.49999985098838806f));
        e = fma2(e, la, f2(1.f));
        e = mul2(e, la);
        a = add2(e, f2(1.f));
    } else {
        la.x = max_nan(la.x, kLeastLog), la.y = max_nan(la.y, kLeastLog);
        // 1.5 2^23 + 127: its sum with a small number is rounded to a whole one, and ends in the bits of 2^n
        constexpr float kBig = 12582912.f + 127.f;
        const float2 t = fma2(la, f2(kLog2e), f2(kBig));
        const float2 y = fma2(add2(t, f2(-kBig)), f2(-0.693147180559945f), la);
        float2 p = fma2(y, f2(0.0013888872927054763f), f2(0.008369109593331814f));
        p = fma2(p, y, f2(0.041667137295007706f));
        p = fma2(p, y, f2(0.16666506230831146f));
        p = fma2(p, y, f2(0.5f));
        p = fma2(p, y, f2(1.f));
        p = mul2(p, y);
        const float2 s =
            make_float2(__uint_as_float(__float_as_uint(t.x) << 23), __uint_as_float(__float_as_uint(t.y) << 23));
        a = fma2(s, p, s);
        e = fma2(s, p, add2(s, f2(-1.f)));
    }
    m = mul2(e, fma2(e, f2(-1.f), f2(-2.f)));  // -e (e + 2)
}

// la a of that a: 0 to fp32 where a is, however far below kLeastLog la lies.
template <bool WIDE>
__device__ __forceinline__ float2 decay_slope2(float2 la, float2 a) {
    if constexpr (WIDE) la.x = max_nan(la.x, kLeastLog), la.y = max_nan(la.y, kLeastLog);
    return mul2(la, a);
}

// sqrt(m)
__device__ __forceinline__ float2 sqrt2(float2 m) {
    float2 r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(m.x));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(m.y));
    return r;
}
// 1 / sqrt(m), finite at m = 0 (where log a, which it meets, is 0 too).
__device__ __forceinline__ float2 rsqrt2(float2 m) {
    m = add2(m, f2(1e-36f));
    return make_float2(rsqrt_approx(m.x), rsqrt_approx(m.y));
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

// One sequence tensor's tokens on their way to shared memory.  LANES lanes are a group with two channels each of
// the strip's and eight tokens; the 32 / LANES groups of a warp lie side by side in its place, [8 tokens]
// [group][2 LANES channels] T, which its lanes fill together, tile after tile, `step` tokens apart: by cp.async
// (waited for with its group, then __syncwarp), or by plain loads where rows start on single
// bf16 elements.  What is not there becomes 0 in tiles that a row ends in.
template <typename T, Rows ROWS, int LANES>
struct Walk {
    static constexpr int kStrip = 2 * LANES, kSub = 32 / LANES, kPlace = kTok * kSub * kStrip;
    static constexpr int kPer = ROWS == kRows16 ? 16 / (int)sizeof(T) : ROWS == kRowsPair ? 2 : 1;  // channels of a copy
    static constexpr int kAcross = kStrip / kPer, kCopies = kPlace / kPer / 32;
    static constexpr int kBytes = kPer * (int)sizeof(T);
    const T* next;  // of this lane's first copy

    // copy k of this lane: its group of the warp, token and channel
    static __device__ __forceinline__ int sub(int lane, int k) { return (lane + 32 * k) / kAcross % kSub; }
    static __device__ __forceinline__ int token(int lane, int k) { return (lane + 32 * k) / (kAcross * kSub); }
    static __device__ __forceinline__ int channel(int lane, int k) { return (lane + 32 * k) % kAcross * kPer; }

    __device__ __forceinline__ void start(const void* base, int64_t row, int64_t stride, int64_t c0, int64_t t, int lane) {
        next = static_cast<const T*>(base) + (row + t + token(lane, 0) + sub(lane, 0) * kTok) * stride + c0 +
               channel(lane, 0);
    }
    // t: the warp's first token; -1: nothing is there.  base: the tensor, for copies of nothing
    __device__ __forceinline__ void fetch(T* place, const void* base, int64_t stride, int t, int n, int step, int have, int lane) {
        if (ROWS != kRowsOne && t >= 0 && t + kTok * kSub <= n) {
            if constexpr (ROWS != kRowsOne) {
                // from copy to copy a fixed number of tokens on (one warp's copies span whole tokens)
                static_assert(32 % (kAcross * kSub) == 0 || kAcross * kSub % 32 == 0, "");
                const uint32_t to = smem_u32(place) + lane * kBytes;
#pragma unroll
                for (int k = 0; k < kCopies; ++k) {
                    const T* from = next + (token(lane, k) - token(lane, 0) + (sub(lane, k) - sub(lane, 0)) * kTok) * stride +
                                    (channel(lane, k) - channel(lane, 0));
                    if (channel(lane, k) < have) {
                        if constexpr (kBytes == 16)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * 32 * kBytes), "l"(from)
                                         : "memory");
                        else
                            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + k * 32 * kBytes),
                                         "l"(from), "n"(kBytes)
                                         : "memory");
                    }
                }
            }
        } else {
            // (copies of single bf16 elements: eight loads at once)
            constexpr int kAtOnce = kCopies < 8 ? kCopies : 8;
#pragma unroll
            for (int k0 = 0; k0 < kCopies; k0 += kAtOnce) {
                T v[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int k = k0 + i, row = token(lane, k) + sub(lane, k) * kTok;
                    const bool live = t >= 0 && t + row < n && channel(lane, k) < have;
                    const T* from = next + (token(lane, k) - token(lane, 0) + (sub(lane, k) - sub(lane, 0)) * kTok) * stride +
                                    (channel(lane, k) - channel(lane, 0));
                    if (!live) from = static_cast<const T*>(base);
                    T* to = place + (lane + 32 * k) * kPer;
                    if constexpr (kBytes == 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from),
                                     "r"(live ? 16 : 0)
                                     : "memory");
                    else if constexpr (kBytes >= 4)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(to)), "l"(from),
                                     "n"(kBytes), "r"(live ? kBytes : 0)
                                     : "memory");
                    else
                        v[i] = live ? *from : from_f32<T>(0.f);
                }
                if constexpr (kBytes < 4) {
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) place[lane + 32 * (k0 + i)] = v[i];
                }
            }
        }
        next += (int64_t)step * stride;
    }
};
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_for() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A pair of channels to memory; `have` of the strip's channels are there.
template <typename T, bool ODD>
__device__ __forceinline__ void store(T* row, float2 v, int lane, int have) {
    if constexpr (!ODD) {
        if (2 * lane < have) *reinterpret_cast<typename Pair<T>::raw*>(row + 2 * lane) = Pair<T>::put(v);
    } else {
        if (2 * lane < have) row[2 * lane] = from_f32<T>(v.x);
        if (2 * lane + 1 < have) row[2 * lane + 1] = from_f32<T>(v.y);
    }
}

// A lane's pairs of channels of a group's tokens, one after another (`step` elements apart).
// ALL: every lane's channels are there.
template <typename T, bool ODD>
struct Rows1 {
    T* to;
    int64_t step;
    __device__ __forceinline__ void start(void* base, int64_t row, int64_t stride, int64_t c0, int64_t t, int lane, int dir) {
        to = static_cast<T*>(base) + (row + t) * stride + c0 + 2 * lane;
        step = dir * stride;
    }
    template <bool ALL>
    __device__ __forceinline__ void put(float2 v, int lane, int have, bool live) {
        if constexpr (ALL && !ODD) {
            *reinterpret_cast<typename Pair<T>::raw*>(to) = Pair<T>::put(v);
        } else {
            if (live) store<T, ODD>(to - 2 * lane, v, lane, have);
        }
        to += step;
    }
};

// fp32 values of a pair of channels, of which `have` of the strip's are there.
__device__ __forceinline__ float2 load_pair(const float* p, int lane, int have) {
    return make_float2(2 * lane < have ? p[2 * lane] : 0.f, 2 * lane + 1 < have ? p[2 * lane + 1] : 0.f);
}

// Blocks of `bytes` of shared memory each that an SM holds at once (of its 228 KB a block takes 1 KB more than it
// asks for), of those `warps` warps of an SM that the registers are for.
constexpr int blocks_of(int warps, int threads, int bytes) {
    const int by_warps = warps * 32 / threads, by_bytes = 228 * 1024 / (bytes + 1024);
    return by_warps < by_bytes ? by_warps : by_bytes;
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

// The same as a message: it counts on `bar` in that block, and nothing waits for what was stored before it, as the
// cluster's barrier does for y on its way to memory (forward, 1 x 4096 x 1024 in bf16: 24 us, with the barrier 28;
// backward, whose registers are all taken, 40 with messages and 34 with the barrier).
__device__ __forceinline__ void send(const void* here, uint64_t* bar, uint32_t rank, float4 v) {
    uint32_t at, count;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(here)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(count) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(count)
                 : "memory");
}
__device__ __forceinline__ void send(const void* here, uint64_t* bar, uint32_t rank, float v) {
    uint32_t at, count;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(here)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(count) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(at), "f"(v), "r"(count)
                 : "memory");
}

// What a block of a cluster needs to take messages: two barriers in turn, and whether a wait has run out (the status word
// says so, and later waits end at once).
struct Mail {
    uint64_t bars[2];
    int abort;
    int pad;
};
__device__ __forceinline__ void open_mail(Mail& m) {  // (a cluster_sync has to follow)
    if (threadIdx.x == 0) {
        mbar_init(&m.bars[0], 1), mbar_init(&m.bars[1], 1);
        fence_barrier_init();
        m.abort = 0;
    }
}
// All threads, after the sends of exchange `count` (from 0): until `bytes` have come to this block.
__device__ __forceinline__ void take_mail(Mail& m, uint32_t count, uint32_t bytes, unsigned int* status) {
    uint64_t* bar = &m.bars[count & 1];
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, bytes);
    if (!mbar_wait(bar, (count >> 1) & 1, &m.abort)) {
        m.abort = 1;
        if (status) atomicExch(status, kStatusTimeout);
    }
}

// How all of a call's rows lie (pointers that are null do not count).
inline Rows rows_of(const void* const* p, const int64_t* strides, int count, int64_t channels, int bytes) {
    uint64_t all = (uint64_t)channels * bytes;
    for (int k = 0; k < count; ++k) all |= reinterpret_cast<uintptr_t>(p[k]) | (uint64_t)strides[k] * bytes;
    return all % 16 == 0 ? kRows16 : all % (2 * bytes) == 0 ? kRowsPair : kRowsOne;
}

// Blocks that split a sequence: eight or four while they are at most three to an SM and have a tile each,
// else one (an exchange between blocks costs more than it gives where strips alone fill half of the GPU).
// 1 x 4096 tokens in bf16, us with 1, 4 and 8.  Forward: 32 strips 50, 28, 24; 64 strips 52, 34, 31 (gated 63, 38, 48);
// 100 strips 52, 38, 44; 128 strips 52, 45, 50 (gated 63, 64, 69).  Backward: 32 strips 104, 46, 34; 64 strips
// 108, 56, 67; 100 strips 112, 65, 71; 128 strips 114, 104, 95.  One rule for both directions and with or without a gate is
// not the best of each: 64 strips forward without a gate lose 3 us by it, 128 strips 7, and 19 backward.
inline int glr_cluster(int64_t strips, int64_t tiles) {
    const int64_t most = 3 * (int64_t)(sm_count() > 0 ? sm_count() : 152);
    if (tiles >= 8 && 8 * strips <= most) return 8;
    return tiles >= 4 && 4 * strips <= most ? 4 : 1;
}

// `beside`: the kernel may start while the one before it ends (of other strips), for whose end it waits before its own.
template <typename Args>
cudaError_t launch_strips(void (*kernel)(Args, int), const Args& a, dim3 grid, int K, int threads, int bytes, bool beside,
                          cudaStream_t st) {
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (K > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)K;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (beside) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, kernel, a, K);
    return launched == cudaSuccess ? cudaGetLastError() : (cudaGetLastError(), launched);
}

// All of a call's strips, `per_row` of each batch row: `one` takes them alone, `some` as clusters.  Where strips are a little
// more than the GPU's places for them, the few that are left over when every SM has as many would keep a few SMs for
// as long as all others: they are split, while the last of the others end (4 x 4096 x 4096 in bf16, gated, backward
// 298 -> 258 us, 8 x 2048 x 2560 155 -> 126, 10 x 1024 x 2048 85 -> 71; but where all have places, 4 x 4096 x 4096,
// 218 -> 241, and where places are taken three times, 16 x 2048 x 4096 forward, 183 -> 196).  As many are split as clusters
// of eight blocks take the places once, three to an SM at least: in fp32 with a gate, backward, where an SM has two places,
// 1 x 4096 x 11200 326 -> 288, on single elements 500 -> 400; 512 strips, 56 left over, 398 -> 418 and 664 -> 600.
template <typename Args>
cudaError_t launch_all(void (*one)(Args, int), void (*some)(Args, int), Args a, int64_t per_row, int per_sm, int threads,
                       int bytes_one, int bytes_some, cudaStream_t st) {
    const int64_t tiles = (a.seqlen + kTile - 1) / kTile, sms = sm_count() > 0 ? sm_count() : 152, places = per_sm * sms;
    const int64_t strips = a.batch * per_row, left = strips % sms;
    const int K = glr_cluster(strips, tiles);
    const int64_t beside = places > 3 * sms ? places : 3 * sms;
    const bool split = strips > places && strips < 2 * places && left > 0 && 8 * left <= beside && tiles >= 16;
    a.first = K > 1 ? 0 : split ? strips - left : strips;
    if (K == 1) {
        const cudaError_t e = launch_strips(one, a, dim3((unsigned)per_row, (unsigned)a.batch), 1, threads, bytes_one, false, st);
        if (e != cudaSuccess || !split) return e;
    }
    const int by = K > 1 ? K : 8;
    return launch_strips(some, a, dim3((unsigned)((strips - a.first) * by)), by, threads, bytes_some, split && K == 1, st);
}

}  // namespace glr
}  // namespace m2
