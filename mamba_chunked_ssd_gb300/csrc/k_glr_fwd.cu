// k_glr_fwd.cu — the gated linear recurrence over whole sequences:
//
//   log a_t = A sigmoid(r_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  y_t = h_t [SiLU(z_t)]
//
// x, r, i [z] are read once and y is written once.  A block walks a strip of 64 channels in
// tiles of 64 tokens; a lane has two channels, a warp eight tokens of the tile.  Each warp
// turns its tokens into factors a and additions u, and the map h -> A h + B of all eight; the
// warps exchange these maps through shared memory, one barrier a tile, and each then runs its
// tokens from the state that enters them.  Inputs come through shared memory, each warp's to its
// own place, tiles ahead.  Where strips are too few to fill the GPU, the blocks of a cluster take a
// sequence's tiles in turn and exchange their tiles' maps through distributed shared memory.
#include "glr_math.cuh"

namespace m2 {
namespace {

using namespace glr;

// Tiles under way ahead of the one that is computed.
template <typename T>
constexpr int kStages = sizeof(T) == 2 ? 3 : 2;

template <typename T, bool GATED>
constexpr int smem_bytes() {
    return kStages<T> * kWarps * (3 + GATED) * kTok * kStrip * (int)sizeof(T) +
           (2 * kWarps + 2 * 8) * 32 * (int)sizeof(float4);
}

template <typename T, Rows ROWS, bool GATED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) k_glr_fwd(const GlrArgs a, int K) {
    constexpr int NT = 3 + GATED, kPlace = kTok * kStrip, S = kStages<T>;
    constexpr bool kOdd = ROWS == kRowsOne;
    using P = Pair<T>;
    using Raw = typename P::raw;
    extern __shared__ __align__(16) uint8_t smem[];
    float4(*sums)[kWarps][32] = reinterpret_cast<float4(*)[kWarps][32]>(smem);
    float4(*parts)[8][32] = reinterpret_cast<float4(*)[8][32]>(smem + 2 * kWarps * 32 * sizeof(float4));
    T* ring = reinterpret_cast<T*>(smem + (2 * kWarps + 2 * 8) * 32 * sizeof(float4));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = K > 1 ? (int)cluster_rank() : 0;
    const int64_t b = blockIdx.y, c0 = (int64_t)(blockIdx.x / K) * kStrip;
    const int have = (int)imin64(a.channels - c0, kStrip);
    const int64_t L = a.seqlen, n = row_length(a.lengths, b, L), tiles = (n + kTile - 1) / kTile;
    const Seq<T> in[4] = {{static_cast<const T*>(a.x) + b * L * a.x_stride + c0, a.x_stride},
                          {static_cast<const T*>(a.r) + b * L * a.r_stride + c0, a.r_stride},
                          {static_cast<const T*>(a.i) + b * L * a.i_stride + c0, a.i_stride},
                          {GATED ? static_cast<const T*>(a.z) + b * L * a.z_stride + c0 : nullptr, a.z_stride}};
    T* y = static_cast<T*>(a.y) + b * L * a.y_stride + c0;
    const float2 A = load_pair(a.A + c0, lane, have);
    float2 carry = a.init ? load_pair(a.init + b * a.channels + c0, lane, have) : f2(0.f);

    auto ahead = [&](int64_t step, int stage) {
        const int64_t t = (step * K + rank) * kTile + warp * kTok;
#pragma unroll
        for (int q = 0; q < NT; ++q)
            fetch<T, ROWS>(ring + ((stage * kWarps + warp) * NT + q) * kPlace, in[q], t, n, have, lane);
        commit();
    };
    if (K > 1) cluster_sync();  // the others' shared memory is there
    for (int s = 0; s < S; ++s) ahead(s, s);
    const int64_t steps = (tiles + K - 1) / K;
    int stage = 0, buf = 0;
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t t = (j * K + rank) * kTile + warp * kTok;
        wait_for<S - 1>();
        __syncwarp();
        const Raw* place = reinterpret_cast<const Raw*>(ring + (stage * kWarps + warp) * NT * kPlace) + lane;
        float2 f[kTok], u[kTok], PA = f2(1.f), PB = f2(0.f);
        Raw z[GATED ? kTok : 1];
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
            const float2 x = P::get(place[k * 32]), r = P::get(place[(kTok + k) * 32]),
                         i = P::get(place[(2 * kTok + k) * 32]);
            if (GATED) z[GATED ? k : 0] = place[(3 * kTok + k) * 32];
            float2 m;
            decay2(mul2(A, sigmoid2(r)), f[k], m);
            u[k] = mul2(mul2(mul2(m, rsqrt2(m)), sigmoid2(i)), x);
        }
        if (t + kTok > n) {  // tokens past the row's end leave the state as it is
#pragma unroll
            for (int k = 0; k < kTok; ++k)
                if (t + k >= n) f[k] = f2(1.f), u[k] = f2(0.f);
        }
#pragma unroll
        for (int k = 0; k < kTok; ++k) PB = fma2(f[k], PB, u[k]), PA = mul2(PA, f[k]);
        sums[buf][warp][lane] = make_float4(PA.x, PA.y, PB.x, PB.y);
        __syncthreads();  // (also: the warp's lanes have read their places)
        ahead(j + S, stage);
        if (++stage == S) stage = 0;

        // the map of the tile's tokens before this warp's, and of the whole tile
        float2 QA = f2(1.f), QB = f2(0.f), h;
        PA = f2(1.f), PB = f2(0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) QA = PA, QB = PB;
            const float4 s = sums[buf][w][lane];
            const float2 sa = make_float2(s.x, s.y);
            PB = fma2(sa, PB, make_float2(s.z, s.w)), PA = mul2(PA, sa);
        }
        if (K == 1) {
            h = carry;
            carry = fma2(PA, carry, PB);
        } else {
            if (warp < K) store_remote(&parts[buf][rank][lane], warp, make_float4(PA.x, PA.y, PB.x, PB.y));
            cluster_sync();
            for (int q = 0; q < K; ++q) {
                if (q == rank) h = carry;
                const float4 s = parts[buf][q][lane];
                carry = fma2(make_float2(s.x, s.y), carry, make_float2(s.z, s.w));
            }
        }
        buf ^= 1;
        if (a.chunk_states && warp == 0 && j * K + rank < tiles)
            store<float, true>(a.chunk_states + (b * ((L + kTile - 1) / kTile) + j * K + rank) * a.channels + c0, h, lane,
                               have);
        h = fma2(QA, h, QB);
        T* row = y + t * a.y_stride;
#pragma unroll
        for (int k = 0; k < kTok; ++k, row += a.y_stride) {
            h = fma2(f[k], h, u[k]);
            float2 o = h;
            if (GATED) {
                const float2 g = P::get(z[GATED ? k : 0]);
                o = mul2(mul2(h, g), sigmoid2(g));
            }
            if (t + k < n) store<T, kOdd>(row, o, lane, have);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (rank == 0 && warp == 0 && a.final_state)
        store<float, true>(a.final_state + b * a.channels + c0, carry, lane, have);
    for (int64_t t = n + rank * kWarps + warp; t < L; t += K * kWarps)
        store<T, kOdd>(y + t * a.y_stride, f2(0.f), lane, have);
    if (a.chunk_states) {
        const int64_t nc = (L + kTile - 1) / kTile;
        for (int64_t g = tiles + rank * kWarps + warp; g < nc; g += K * kWarps)
            store<float, true>(a.chunk_states + (b * nc + g) * a.channels + c0, carry, lane, have);
    }
}

template <typename T, Rows ROWS, bool GATED>
cudaError_t launch(const GlrArgs& a, cudaStream_t st) {
    constexpr int bytes = smem_bytes<T, GATED>();
    const int64_t strips = (a.channels + kStrip - 1) / kStrip, tiles = (a.seqlen + kTile - 1) / kTile;
    const int K = glr_cluster(strips * a.batch, tiles);
    return launch_strips(k_glr_fwd<T, ROWS, GATED>, a, strips, K, bytes, st);
}

template <typename T>
cudaError_t launch_t(const GlrArgs& a, cudaStream_t st) {
    const void* p[] = {a.x, a.r, a.i, a.z, a.y};
    const int64_t strides[] = {a.x_stride, a.r_stride, a.i_stride, a.z ? a.z_stride : 0, a.y_stride};
    switch (rows_of(p, strides, 5, a.channels, sizeof(T))) {
        case kRows16: return a.z ? launch<T, kRows16, true>(a, st) : launch<T, kRows16, false>(a, st);
        case kRowsPair: return a.z ? launch<T, kRowsPair, true>(a, st) : launch<T, kRowsPair, false>(a, st);
        default: return a.z ? launch<T, kRowsOne, true>(a, st) : launch<T, kRowsOne, false>(a, st);
    }
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
