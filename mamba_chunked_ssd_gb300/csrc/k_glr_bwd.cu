// k_glr_bwd.cu — gradients of the gated linear recurrence.  With v = sigmoid(i) x,
// s = sqrt(1 - a^2) and la = log a:
//
//   dh_t = dy_t [SiLU(z_t)] + a_{t+1} dh_{t+1}          dz = dy h SiLU'(z)
//   dx   = dh s sigmoid(i)                              di = dx x (1 - sigmoid(i))
//   E    = la dL/dla = dh (la a h_{t-1} - la a^2 / s v) dr = E (1 - sigmoid(r)),  dA = sum E / A
//
// (la / s is finite where s vanishes, d la is not.)  Everything is read once and written once:
// a block walks its strip of 64 channels backwards in tiles of 64 tokens, a warp with eight
// tokens of each.  The states inside a tile come from the chunk state that enters it, which the forward
// pass kept, by the same exchange of maps as there; the maps of the gradients, c -> A (c + ..)
// from the other end, go through the same barrier.  What both halves need stays in
// registers, or in the places of inputs that have been used.
#include "glr_math.cuh"

namespace m2 {
namespace {

using namespace glr;

constexpr int kStages = 2;

template <typename T, bool GATED>
constexpr int smem_bytes() {
    return kStages * kWarps * (4 + GATED) * kTok * kStrip * (int)sizeof(T) +
           2 * kWarps * 32 * (int)(sizeof(float4) + sizeof(float2)) + 2 * 8 * 32 * (int)sizeof(float4) +
           (GATED && sizeof(T) == 2 ? kThreads * kTok * (int)sizeof(float2) : 0);
}

// Two fp32 values in the places of two raw pairs (one of them where a raw pair is fp32).
__device__ __forceinline__ void stash(uint32_t* p, uint32_t* q, float2 v) {
    *p = __float_as_uint(v.x), *q = __float_as_uint(v.y);
}
__device__ __forceinline__ float2 unstash(const uint32_t* p, const uint32_t* q) {
    return make_float2(__uint_as_float(*p), __uint_as_float(*q));
}
__device__ __forceinline__ void stash(float2* p, float2*, float2 v) { *p = v; }
__device__ __forceinline__ float2 unstash(const float2* p, const float2*) { return *p; }

template <typename T, Rows ROWS, bool GATED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) k_glr_bwd(const GlrBwdArgs a, int K) {
    constexpr int NT = 4 + GATED, kPlace = kTok * kStrip, S = kStages;
    constexpr bool kOdd = ROWS == kRowsOne;
    using P = Pair<T>;
    using Raw = typename P::raw;
    extern __shared__ __align__(16) uint8_t smem[];
    float4(*sums)[kWarps][32] = reinterpret_cast<float4(*)[kWarps][32]>(smem);
    float4(*parts)[8][32] = reinterpret_cast<float4(*)[8][32]>(smem + 2 * kWarps * 32 * sizeof(float4));
    float2(*rsums)[kWarps][32] =
        reinterpret_cast<float2(*)[kWarps][32]>(smem + (2 * kWarps + 2 * 8) * 32 * sizeof(float4));
    uint8_t* rest = smem + (2 * kWarps + 2 * 8) * 32 * sizeof(float4) + 2 * kWarps * 32 * sizeof(float2);
    T* ring = reinterpret_cast<T*>(rest);
    // the factors of dz, where z's places do not hold them
    float2* dzs = reinterpret_cast<float2*>(rest + kStages * kWarps * NT * kPlace * sizeof(T)) + threadIdx.x;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = K > 1 ? (int)cluster_rank() : 0;
    const int64_t b = blockIdx.y, c0 = (int64_t)(blockIdx.x / K) * kStrip;
    const int have = (int)imin64(a.channels - c0, kStrip);
    const int64_t L = a.seqlen, n = row_length(a.lengths, b, L), tiles = (n + kTile - 1) / kTile;
    const Seq<T> in[5] = {{static_cast<const T*>(a.x) + b * L * a.x_stride + c0, a.x_stride},
                          {static_cast<const T*>(a.r) + b * L * a.r_stride + c0, a.r_stride},
                          {static_cast<const T*>(a.i) + b * L * a.i_stride + c0, a.i_stride},
                          {static_cast<const T*>(a.dy) + b * L * a.dy_stride + c0, a.dy_stride},
                          {GATED ? static_cast<const T*>(a.z) + b * L * a.z_stride + c0 : nullptr, a.z_stride}};
    T* dx = static_cast<T*>(a.dx) + b * L * a.dx_stride + c0;
    T* dr = static_cast<T*>(a.dr) + b * L * a.dr_stride + c0;
    T* di = static_cast<T*>(a.di) + b * L * a.di_stride + c0;
    T* dz = GATED ? static_cast<T*>(a.dz) + b * L * a.dz_stride + c0 : nullptr;
    const float* states = a.chunk_states + b * ((L + kTile - 1) / kTile) * a.channels + c0;
    const float2 A = load_pair(a.A + c0, lane, have);
    float2 carry = a.dfinal ? load_pair(a.dfinal + b * a.channels + c0, lane, have) : f2(0.f);
    float2 total = f2(0.f);

    // the tile of a step (below 0: none) and this warp's first token in it
    auto tile_of = [&](int64_t step) { return tiles - 1 - (step * K + rank); };
    auto ahead = [&](int64_t step, int stage) {
        const int64_t g = tile_of(step), t = (g < 0 ? 0 : g) * kTile + warp * kTok;
#pragma unroll
        for (int q = 0; q < NT; ++q)
            fetch<T, ROWS>(ring + ((stage * kWarps + warp) * NT + q) * kPlace, in[q], t, g < 0 ? 0 : n, have, lane);
        commit();
    };
    if (K > 1) cluster_sync();  // the others' shared memory is there
    for (int s = 0; s < S; ++s) ahead(s, s);
    const int64_t steps = (tiles + K - 1) / K;
    int stage = 0, buf = 0;
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t g = tile_of(j), t = (g < 0 ? 0 : g) * kTile + warp * kTok;
        const int live = g < 0 ? 0 : (int)imin64(n - t < 0 ? 0 : n - t, kTok);  // this warp's tokens
        float2 h = g < 0 ? f2(0.f) : load_pair(states + g * a.channels, lane, have);
        wait_for<S - 1>();
        __syncwarp();
        Raw* px = reinterpret_cast<Raw*>(ring + (stage * kWarps + warp) * NT * kPlace) + lane;
        Raw *pr = px + kTok * 32, *pi = px + 2 * kTok * 32, *pd = px + 3 * kTok * 32, *pz = px + 4 * kTok * 32;
        float2 f[kTok], s[kTok], c2[kTok], oi[kTok];  // a; s sigmoid(i); -la a^2 / s v; 1 - sigmoid(i)
        float2 PA = f2(1.f), PB = f2(0.f), PR = f2(0.f);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const float2 x = P::get(px[k * 32]);
            float2 sr = sigmoid2(P::get(pr[k * 32]));
            const float2 si = sigmoid2(P::get(pi[k * 32]));
            const float2 la = mul2(A, sr);
            float2 m;
            decay2(la, f[k], m);
            const float2 q = rsqrt2(m);
            s[k] = mul2(mul2(m, q), si);
            oi[k] = fma2(si, f2(-1.f), f2(1.f));
            const float2 ap = mul2(f[k], q);
            c2[k] = mul2(mul2(mul2(mul2(ap, ap), mul2(la, f2(-1.f))), s[k]), x);
            float2 gy = P::get(pd[k * 32]);
            if (GATED) {
                const float2 z = P::get(pz[k * 32]), sz = sigmoid2(z);
                const float2 d = mul2(gy, sz);
                gy = mul2(d, z);
                const float2 dzc = fma2(gy, fma2(sz, f2(-1.f), f2(1.f)), d);
                stash(pd + k * 32, pz + k * 32, gy);
                if (sizeof(T) == 2) dzs[k * kThreads] = dzc;
                else *reinterpret_cast<float2*>(pz + k * 32) = dzc;
            }
            if (k >= live) f[k] = f2(1.f), s[k] = c2[k] = sr = gy = f2(0.f);
            stash(pr + k * 32, pi + k * 32, sr);
            PB = fma2(f[k], PB, mul2(s[k], x));
            PA = mul2(PA, f[k]);
            PR = fma2(PA, gy, PR);
        }
        sums[buf][warp][lane] = make_float4(PA.x, PA.y, PB.x, PB.y);
        rsums[buf][warp][lane] = PR;
        __syncthreads();
        // the state before this warp's tokens
        for (int w = 0; w < warp; ++w) {
            const float4 v = sums[buf][w][lane];
            h = fma2(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
        }
        // the gradient map of the tile's tokens behind this warp's, and of the whole tile
        float2 QA = f2(1.f), QR = f2(0.f), c;
        PA = f2(1.f), PR = f2(0.f);
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            if (w == warp) QA = PA, QR = PR;
            const float2 fa = *reinterpret_cast<const float2*>(&sums[buf][w][lane]);
            PR = fma2(fa, PR, rsums[buf][w][lane]), PA = mul2(PA, fa);
        }
        if (K == 1) {
            c = carry;
            carry = fma2(PA, carry, PR);
        } else {
            if (warp < K) store_remote(&parts[buf][rank][lane], warp, make_float4(PA.x, PA.y, PR.x, PR.y));
            cluster_sync();
            for (int q = 0; q < K; ++q) {
                if (q == rank) c = carry;
                const float4 v = parts[buf][q][lane];
                carry = fma2(make_float2(v.x, v.y), carry, make_float2(v.z, v.w));
            }
        }
        c = fma2(QA, c, QR);
        buf ^= 1;

        float2 hp[kTok];  // the state before each token
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            hp[k] = h;
            h = fma2(f[k], h, mul2(s[k], P::get(px[k * 32])));
            if (GATED) {
                const float2 dzc = sizeof(T) == 2 ? dzs[k * kThreads] : *reinterpret_cast<const float2*>(pz + k * 32);
                if (k < live) store<T, kOdd>(dz + (t + k) * a.dz_stride, mul2(dzc, h), lane, have);
            }
        }
        float2 e8 = f2(0.f);
#pragma unroll
        for (int k = kTok - 1; k >= 0; --k) {
            float2 dh = GATED ? unstash(pd + k * 32, pz + k * 32) : P::get(pd[k * 32]);
            if (k >= live) dh = f2(0.f);
            dh = add2(dh, c);
            const float2 sr = unstash(pr + k * 32, pi + k * 32);
            const float2 e = mul2(dh, fma2(mul2(mul2(A, sr), f[k]), hp[k], c2[k]));
            e8 = add2(e8, e);
            const float2 gx = mul2(dh, s[k]);
            c = mul2(f[k], dh);
            if (k < live) {
                store<T, kOdd>(dx + (t + k) * a.dx_stride, gx, lane, have);
                store<T, kOdd>(dr + (t + k) * a.dr_stride, mul2(e, fma2(sr, f2(-1.f), f2(1.f))), lane, have);
                store<T, kOdd>(di + (t + k) * a.di_stride, mul2(mul2(gx, P::get(px[k * 32])), oi[k]), lane, have);
            }
        }
        total = add2(total, e8);
        __syncwarp();  // the places have been read
        ahead(j + S, stage);
        if (++stage == S) stage = 0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (rank == 0 && warp == 0 && a.dinit) store<float, true>(a.dinit + b * a.channels + c0, carry, lane, have);
    for (int64_t t = n + rank * kWarps + warp; t < L; t += K * kWarps) {
        store<T, kOdd>(dx + t * a.dx_stride, f2(0.f), lane, have);
        store<T, kOdd>(dr + t * a.dr_stride, f2(0.f), lane, have);
        store<T, kOdd>(di + t * a.di_stride, f2(0.f), lane, have);
        if (GATED) store<T, kOdd>(dz + t * a.dz_stride, f2(0.f), lane, have);
    }
    __syncthreads();
    rsums[0][warp][lane] = total;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) total = add2(total, rsums[0][w][lane]);
        store<float, true>(a.partials + (b * K + rank) * a.channels + c0, total, lane, have);
    }
}

int64_t strips_of(int64_t channels) { return (channels + kStrip - 1) / kStrip; }

template <typename T, Rows ROWS, bool GATED>
cudaError_t launch(const GlrBwdArgs& a, cudaStream_t st) {
    constexpr int bytes = smem_bytes<T, GATED>();
    const int64_t strips = strips_of(a.channels);
    const int K = glr_cluster(strips * a.batch, (a.seqlen + kTile - 1) / kTile);
    const cudaError_t e = launch_strips(k_glr_bwd<T, ROWS, GATED>, a, strips, K, bytes, st);
    if (e != cudaSuccess) return e;
    return launch_sum_rows(a.partials, a.batch * K, {a.dA, a.channels}, {}, {}, a.A, st);
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

int64_t glr_bwd_partials(int64_t batch, int64_t seqlen, int64_t channels) {
    return batch * glr_cluster(strips_of(channels) * batch, (seqlen + kTile - 1) / kTile);
}

cudaError_t launch_glr_bwd(const GlrBwdArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
