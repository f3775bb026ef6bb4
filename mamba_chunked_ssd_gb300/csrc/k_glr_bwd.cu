// k_glr_bwd.cu — gradients of the gated linear recurrence.  With v = sigmoid(i) x,
// s = sqrt(1 - a^2) and la = log a:
//
//   dh_t = dy_t [SiLU(z_t)] + a_{t+1} dh_{t+1}          dz = dy h SiLU'(z)
//   dx   = dh s sigmoid(i)                              di = dx x (1 - sigmoid(i))
//   E    = la dL/dla = dh la a (h_{t-1} - a / s v)     dr = E (1 - sigmoid(r)),  dA = sum E / A
//
// (la / s is finite where s vanishes, dL/dla is not.)  Everything is read once and written once:
// a block walks its strip of 32 channels backwards in tiles of 64 tokens, a group of 16 lanes with eight
// tokens of each.  The states inside a tile come from the chunk state that enters it, which the forward
// pass kept, by the same exchange of maps as there; the maps of the gradients, c -> A c + R
// from the other end, go through the same barrier.  What both halves need stays in
// registers or in shared memory, in the places of inputs that have been used where they fit.
// About 60 instructions an element, and 16 (gated 12) warps of an SM that wait for one another at each tile's exchange: neither
// the issue slots (55 % of them, gated) nor DRAM (61 %) are full, three or four warps to a scheduler are what bounds
// it.  16 x 1024 x 4096 in bf16 196 us, 4.8 TB/s, gated 243 us, 5.0 TB/s; 4 x 4096 x 4096 216 us, gated 258; in fp32 326 us,
// gated, with 8 warps, 417.
#include <type_traits>

#include "glr_math.cuh"

namespace m2 {
namespace {

using namespace glr;

constexpr int kStages = 2;
constexpr int kLanes = 16;
// Warps of an SM that the registers are for: as many as shared memory allows, too, but in fp32 with a gate (4 x 4096 x 4096
// in bf16: with 16 220 us, with 12 of more registers each 259; gated, where 16 do not fit, 298).
template <typename T, bool GATED>
constexpr int kWarpsOf = sizeof(T) == 2 && !GATED ? 16 : 12;

template <typename T, bool GATED, int LANES>
constexpr int smem_bytes(bool cluster) {
    return kStages * kGroups * LANES * 2 * (4 + GATED) * kTok * (int)sizeof(T) +
           (4 * kGroups + (cluster ? 2 * 8 : 0)) * LANES * (int)sizeof(float4) +
           (sizeof(T) == 2 ? (2 + GATED) * kGroups * LANES * kTok * (int)sizeof(float2) : 0);
}
// Blocks of an SM: four of bf16 without a gate, else three, two of fp32 with a gate.
template <typename T, bool GATED, int LANES>
constexpr int kBlocks = blocks_of(kWarpsOf<T, GATED>, kGroups* LANES, smem_bytes<T, GATED, LANES>(false));

// Two fp32 values in the places of two raw pairs (one of them where a raw pair is fp32).
__device__ __forceinline__ void stash(uint32_t* p, uint32_t* q, float2 v) {
    *p = __float_as_uint(v.x), *q = __float_as_uint(v.y);
}
__device__ __forceinline__ float2 unstash(const uint32_t* p, const uint32_t* q) {
    return make_float2(__uint_as_float(*p), __uint_as_float(*q));
}
__device__ __forceinline__ void stash(float2* p, float2*, float2 v) { *p = v; }
__device__ __forceinline__ float2 unstash(const float2* p, const float2*) { return *p; }

template <typename T, Rows ROWS, bool GATED, int LANES, bool CLUSTER>
__global__ void __launch_bounds__(kGroups* LANES, kBlocks<T, GATED, LANES>) k_glr_bwd(const GlrBwdArgs a, int K) {
    using W = Walk<T, ROWS, LANES>;
    constexpr int NT = 4 + GATED, S = kStages, kSub = W::kSub, kPlace = W::kPlace, kStrip = W::kStrip;
    constexpr int kWarps = kGroups / kSub, kThreads = kGroups * LANES;
    constexpr bool kOdd = ROWS == kRowsOne;
    using P = Pair<T>;
    using Raw = typename P::raw;
    extern __shared__ __align__(16) uint8_t smem[];
    using Maps = float4[kGroups][LANES];
    Maps* sums = reinterpret_cast<Maps*>(smem);   // of the states
    Maps* rsums = sums + 2;                       // of the gradients
    float4(*parts)[8][LANES] = reinterpret_cast<float4(*)[8][LANES]>(rsums + 2);
    T* ring = reinterpret_cast<T*>(parts + (CLUSTER ? 2 : 0));
    // what does not fit where bf16 inputs lay: each thread's uo, w and factors of dz
    float2* kept = reinterpret_cast<float2*>(ring + S * kWarps * NT * kPlace) + threadIdx.x;
    if (!CLUSTER) K = 1;
    const int warp = threadIdx.x / 32, group = threadIdx.x / LANES, lane = threadIdx.x % LANES, wl = threadIdx.x % 32;
    const int rank = CLUSTER ? (int)cluster_rank() : 0;
    // the strip and its batch row: of the grid's two dimensions, or counted through all rows
    int64_t b = blockIdx.y, c0 = (int64_t)blockIdx.x * kStrip;
    if constexpr (CLUSTER) {
        const int64_t per_row = (a.channels + kStrip - 1) / kStrip, strip = a.first + blockIdx.x / K;
        b = strip / per_row, c0 = strip % per_row * kStrip;
    } else if (b * gridDim.x + blockIdx.x >= a.first) {
        return;  // (the clusters take those)
    }
    const int have = (int)imin64(a.channels - c0, kStrip);
    const int L = (int)a.seqlen, n = __shfl_sync(0xffffffffu, (int)row_length(a.lengths, b, L), 0), tiles = (n + kTile - 1) / kTile;
    const int step = K * kTile;
    int g = tiles - 1 - rank;                              // the tile that is computed (below 0: none)
    int ta = g * kTile + warp * kSub * kTok;               // the warp's first token of the tile that is fetched
    W in[NT];
    in[0].start(a.x, b * L, a.x_stride, c0, ta, wl);
    in[1].start(a.r, b * L, a.r_stride, c0, ta, wl);
    in[2].start(a.i, b * L, a.i_stride, c0, ta, wl);
    in[3].start(a.dy, b * L, a.dy_stride, c0, ta, wl);
    if (GATED) in[NT - 1].start(a.z, b * L, a.z_stride, c0, ta, wl);
    T* dx = static_cast<T*>(a.dx) + b * L * a.dx_stride + c0;
    T* dr = static_cast<T*>(a.dr) + b * L * a.dr_stride + c0;
    T* di = static_cast<T*>(a.di) + b * L * a.di_stride + c0;
    T* dz = GATED ? static_cast<T*>(a.dz) + b * L * a.dz_stride + c0 : nullptr;
    const float* states = a.chunk_states + (b * ((L + kTile - 1) / kTile)) * a.channels + c0;
    const float2 A = load_pair(a.A + c0, lane, have);
    float2 carry = a.dfinal ? load_pair(a.dfinal + b * a.channels + c0, lane, have) : f2(0.f);
    float2 total = f2(0.f);
    const int64_t strides[5] = {a.x_stride, a.r_stride, a.i_stride, a.dy_stride, a.z_stride};
    const void* bases[5] = {a.x, a.r, a.i, a.dy, a.z};
    auto ahead = [&](int stage) {
#pragma unroll
        for (int q = 0; q < NT; ++q)
            in[q].fetch(ring + ((stage * kWarps + warp) * NT + q) * kPlace, bases[q], strides[q], ta, n, -step, have, wl);
        ta = ta < 0 ? -1 : ta - step;
        commit();
    };
    griddep_launch_dependents();  // (what is launched beside this takes other strips, or waits for this grid's end)
    if (CLUSTER) cluster_sync();  // the others' shared memory is there
    for (int s = 0; s < S; ++s) ahead(s);
    const int steps = (tiles + K - 1) / K;
    int buf = 0;
    auto walk = [&](auto wide) {
        int stage = 0;
        float2 before = g < 0 ? f2(0.f) : load_pair(states + (int64_t)g * a.channels, lane, have);
        for (int j = 0; j < steps; ++j, g -= K) {
            const int t = g * kTile + group * kTok;
            const int live = g < 0 ? 0 : min(max(n - t, 0), kTok);  // this group's tokens
            float2 h = before;  // the state that enters the tile; the next one's is on its way
            if (g >= K) before = load_pair(states + (int64_t)(g - K) * a.channels, lane, have);
            wait_for<S - 1>();
            __syncwarp();
            Raw* px = reinterpret_cast<Raw*>(ring + (stage * kWarps + warp) * NT * kPlace) + wl;
            Raw *pr = px + kTok * 32, *pi = px + 2 * kTok * 32, *pd = px + 3 * kTok * 32, *pz = px + 4 * kTok * 32;
            // The second half needs a, s sigmoid(i), u = s v; sigmoid(r), u (1 - sigmoid(i)), a v / s, and the
            // gradient of h; the latter lie in shared memory (registers for them would leave too few warps).
            auto keep = [&](Raw* at, int which, int k, float2 v) {
                if constexpr (sizeof(T) == 2) kept[(which * kTok + k) * kThreads] = v;
                else *reinterpret_cast<float2*>(at + k * 32) = v;
            };
            auto take = [&](const Raw* at, int which, int k) {
                if constexpr (sizeof(T) == 2) return kept[(which * kTok + k) * kThreads];
                else return *reinterpret_cast<const float2*>(at + k * 32);
            };
            float2 f[kTok], s[kTok], u[kTok];
            float2 PA = f2(1.f), PB = f2(0.f), PR = f2(0.f);
            auto factors = [&](auto whole) {
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    const float2 x = P::get(px[k * 32]);
                    float2 sr = sigmoid2(P::get(pr[k * 32]));
                    const float2 si = sigmoid2(P::get(pi[k * 32])), v = mul2(si, x);
                    float2 m;
                    decay2<decltype(wide)::value>(mul2(A, sr), f[k], m);
                    const float2 q = rsqrt2(m), mq = mul2(m, q);
                    s[k] = mul2(mq, si);
                    u[k] = mul2(mq, v);
                    float2 w = mul2(mul2(f[k], q), v);
                    float2 gy = P::get(pd[k * 32]);
                    if (GATED) {
                        const float2 z = P::get(pz[k * 32]), sz = sigmoid2(z);
                        const float2 d = mul2(gy, sz);
                        gy = mul2(d, z);
                        const float2 dzc = fma2(gy, fma2(sz, f2(-1.f), f2(1.f)), d);
                        stash(pd + k * 32, pz + k * 32, gy);
                        keep(pz, 2, k, dzc);
                    }
                    if (!decltype(whole)::value && k >= live) f[k] = f2(1.f), s[k] = u[k] = w = sr = gy = f2(0.f);
                    keep(px, 0, k, fma2(mul2(u[k], f2(-1.f)), si, u[k]));
                    stash(pr + k * 32, pi + k * 32, sr);
                    keep(pi, 1, k, w);
                    PB = fma2(f[k], PB, u[k]);
                    PA = mul2(PA, f[k]);
                    PR = fma2(PA, gy, PR);
                }
            };
            if (live == kTok) factors(std::true_type{});
            else factors(std::false_type{});
            sums[buf][group][lane] = make_float4(PA.x, PA.y, PB.x, PB.y);
            rsums[buf][group][lane] = make_float4(PA.x, PA.y, PR.x, PR.y);
            __syncthreads();
            // the state before this group's tokens
#pragma unroll
            for (int w = 0; w < kGroups - 1; ++w)
                if (w < group) {
                    const float4 v = sums[buf][w][lane];
                    h = fma2(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
                }
            // the gradient that comes back to its last one, and the one that leaves the tile
            float2 c = carry;
            if constexpr (CLUSTER) {
                PA = f2(1.f), PR = f2(0.f);
#pragma unroll
                for (int w = kGroups - 1; w >= 0; --w) {
                    const float4 v = rsums[buf][w][lane];
                    const float2 fa = make_float2(v.x, v.y);
                    PR = fma2(fa, PR, make_float2(v.z, v.w)), PA = mul2(PA, fa);
                }
                if (group < K) store_remote(&parts[buf][rank][lane], group, make_float4(PA.x, PA.y, PR.x, PR.y));
                cluster_sync();
                for (int q = 0; q < K; ++q) {
                    if (q == rank) c = carry;
                    const float4 v = parts[buf][q][lane];
                    carry = fma2(make_float2(v.x, v.y), carry, make_float2(v.z, v.w));
                }
#pragma unroll
                for (int w = kGroups - 1; w > 0; --w)
                    if (w > group) {
                        const float4 v = rsums[buf][w][lane];
                        c = fma2(make_float2(v.x, v.y), c, make_float2(v.z, v.w));
                    }
            } else {
#pragma unroll
                for (int w = kGroups - 1; w >= 0; --w) {
                    if (w == group) c = carry;
                    const float4 v = rsums[buf][w][lane];
                    carry = fma2(make_float2(v.x, v.y), carry, make_float2(v.z, v.w));
                }
            }
            buf ^= 1;

            Rows1<T, kOdd> ox, orr, oi, oz;
            if (GATED) oz.start(a.dz, b * L, a.dz_stride, c0, t, lane, 1);
            ox.start(a.dx, b * L, a.dx_stride, c0, t + kTok - 1, lane, -1);
            orr.start(a.dr, b * L, a.dr_stride, c0, t + kTok - 1, lane, -1);
            oi.start(a.di, b * L, a.di_stride, c0, t + kTok - 1, lane, -1);
            float2 e8 = f2(0.f);
            auto tokens = [&](auto all) {
                constexpr bool kAll = decltype(all)::value;
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    const float2 last = h;
                    h = fma2(f[k], h, u[k]);
                    u[k] = last;
                    if (GATED) oz.template put<kAll>(mul2(take(pz, 2, k), h), lane, have, k < live);
                }
#pragma unroll
                for (int k = kTok - 1; k >= 0; --k) {
                    float2 dh = GATED ? unstash(pd + k * 32, pz + k * 32) : P::get(pd[k * 32]);
                    if (!kAll && k >= live) dh = f2(0.f);
                    dh = add2(dh, c);
                    const float2 sr = unstash(pr + k * 32, pi + k * 32);
                    const float2 slope = decay_slope2<decltype(wide)::value>(mul2(A, sr), f[k]);
                    float2 e = mul2(mul2(dh, slope), fma2(take(pi, 1, k), f2(-1.f), u[k]));
                    if (!kAll && k >= live) e = f2(0.f);  // (0 A is not a number where A is -infinity)
                    e8 = add2(e8, e);
                    c = mul2(f[k], dh);
                    ox.template put<kAll>(mul2(dh, s[k]), lane, have, k < live);
                    orr.template put<kAll>(fma2(mul2(e, f2(-1.f)), sr, e), lane, have, k < live);
                    oi.template put<kAll>(mul2(dh, take(px, 0, k)), lane, have, k < live);
                }
            };
            if (live == kTok && have == kStrip) tokens(std::true_type{});
            else tokens(std::false_type{});
            total = add2(total, e8);
            __syncwarp();  // the places have been read
            ahead(stage);
            if (++stage == S) stage = 0;
        }
    };
    if (__syncthreads_and(A.x >= -1.f && A.y >= -1.f)) walk(std::false_type{});
    else walk(std::true_type{});
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (rank == 0 && group == 0 && a.dinit) store<float, true>(a.dinit + b * a.channels + c0, carry, lane, have);
    for (int64_t t = n + rank * kGroups + group; t < L; t += K * kGroups) {
        store<T, kOdd>(dx + t * a.dx_stride, f2(0.f), lane, have);
        store<T, kOdd>(dr + t * a.dr_stride, f2(0.f), lane, have);
        store<T, kOdd>(di + t * a.di_stride, f2(0.f), lane, have);
        if (GATED) store<T, kOdd>(dz + t * a.dz_stride, f2(0.f), lane, have);
    }
    // the blocks' parts of A dA, in the order of their groups and ranks
    __syncthreads();
    float2* part = reinterpret_cast<float2*>(smem) + lane;
    part[group * LANES] = total;
    __syncthreads();
    if (group == 0) {
#pragma unroll
        for (int w = 1; w < kGroups; ++w) total = add2(total, part[w * LANES]);
    }
    if constexpr (CLUSTER) {
        // (the places that the last step did not use: the first block may still be reading those)
        if (group == 0) store_remote(&parts[buf][rank][lane], 0, make_float4(total.x, total.y, 0.f, 0.f));
        cluster_sync();
        if (rank == 0 && group == 0) {
            total = f2(0.f);
            for (int q = 0; q < K; ++q) total = add2(total, make_float2(parts[buf][q][lane].x, parts[buf][q][lane].y));
        }
    }
    if (rank == 0 && group == 0) store<float, true>(a.partials + b * a.channels + c0, total, lane, have);
    if (CLUSTER) griddep_wait();
}

template <typename T, Rows ROWS, bool GATED>
cudaError_t launch(const GlrBwdArgs& a, cudaStream_t st) {
    const int64_t per_row = (a.channels + 2 * kLanes - 1) / (2 * kLanes);
    const cudaError_t e =
        launch_all(k_glr_bwd<T, ROWS, GATED, kLanes, false>, k_glr_bwd<T, ROWS, GATED, kLanes, true>, a, per_row,
                   kBlocks<T, GATED, kLanes>, kGroups * kLanes, smem_bytes<T, GATED, kLanes>(false),
                   smem_bytes<T, GATED, kLanes>(true), st);
    if (e != cudaSuccess) return e;
    return launch_sum_rows(a.partials, a.batch, {a.dA, a.channels}, {}, {}, a.A, st);
}

template <typename T>
cudaError_t launch_t(const GlrBwdArgs& a, cudaStream_t st) {
    const void* p[] = {a.x, a.r, a.i, a.dy, a.dx, a.dr, a.di, a.z, a.dz};
    const int64_t strides[] = {a.x_stride,  a.r_stride,  a.i_stride,           a.dy_stride,         a.dx_stride,
                               a.dr_stride, a.di_stride, a.z ? a.z_stride : 0, a.z ? a.dz_stride : 0};
    switch (rows_of(p, strides, 9, a.channels, sizeof(T))) {
        case kRows16: return a.z ? launch<T, kRows16, true>(a, st) : launch<T, kRows16, false>(a, st);
        case kRowsPair: return a.z ? launch<T, kRowsPair, true>(a, st) : launch<T, kRowsPair, false>(a, st);
        default: return a.z ? launch<T, kRowsOne, true>(a, st) : launch<T, kRowsOne, false>(a, st);
    }
}

}  // namespace

cudaError_t launch_glr_bwd(const GlrBwdArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
