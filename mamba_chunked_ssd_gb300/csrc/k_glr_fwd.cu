// k_glr_fwd.cu — the gated linear recurrence over whole sequences:
//
//   log a_t = A sigmoid(r_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  y_t = h_t [SiLU(z_t)]
//
// x, r, i [z] are read once and y is written once.  A block walks a strip of 32 channels in
// tiles of 64 tokens: 8 groups of 16 lanes, two channels to a lane, eight tokens to a group.  A
// group turns its tokens into factors a and additions u, and the map h -> A h + B of all eight;
// the groups exchange these maps through shared memory, one barrier a tile, and each then runs its
// tokens from the state that enters them.  Inputs come through shared memory, each warp's to its own
// place, tiles ahead.  Where strips are too few to fill the GPU, the blocks of a cluster take a
// sequence's tiles in turn and send one another their tiles' maps.
// About 32 instructions an element (a third of them the gates', the rest the decay's, the exchange's and
// the loads') leave 60 % of the issue slots used by 16 warps of 128 registers: that is what bounds it next to
// memory.  16 x 2048 x 4096 in bf16: 183 us, 5.9 TB/s; 4 x 8192 x 4096, 512 strips of which some SMs have three
// and some four: 214 us, 5.0 TB/s.  In fp32 4 x 4096 x 4096 173 us, 6.2 TB/s, gated 214.  Rows on pairs take copies of four
// bytes and spill registers, one block a strip: 4 x 8192 x 4090 in bf16 756 us.
#include <type_traits>

#include "glr_math.cuh"

namespace m2 {
namespace {

using namespace glr;

// Tiles under way ahead of the one that is computed, lanes of a group, and warps of an SM.  4 x 8192 x 4096 /
// 16 x 2048 x 4096 in bf16: 214 / 183 us; strips of 64 channels (32 lanes) 230 / 200, of 16 channels
// 255 / 233 (rows of 32 bytes); two stages 216 / 190; 20 warps of fewer registers 224 / 188, 24 282 / 237.
template <typename T>
constexpr int kStages = sizeof(T) == 2 ? 3 : 2;
constexpr int kLanes = 16;
constexpr int kWarpsOf = 16;

template <typename T, bool GATED, int LANES>
constexpr int smem_bytes(bool cluster) {
    return kStages<T> * kGroups * LANES * 2 * (3 + GATED) * kTok * (int)sizeof(T) +
           (2 * kGroups + (cluster ? 2 * 8 : 0)) * LANES * (int)sizeof(float4) + (cluster ? (int)sizeof(Mail) + 8 : 0);
}
// Four blocks of an SM, three of fp32 with a gate.
template <typename T, bool GATED, int LANES>
constexpr int kBlocks = blocks_of(kWarpsOf, kGroups* LANES, smem_bytes<T, GATED, LANES>(false));

// CLUSTER: K blocks take a sequence's tiles in turn, else K is 1.
template <typename T, Rows ROWS, bool GATED, int LANES, bool CLUSTER>
__global__ void __launch_bounds__(kGroups* LANES, kBlocks<T, GATED, LANES>) k_glr_fwd(const GlrArgs a, int K) {
    using W = Walk<T, ROWS, LANES>;
    constexpr int NT = 3 + GATED, S = kStages<T>, kSub = W::kSub, kPlace = W::kPlace, kStrip = W::kStrip;
    constexpr int kWarps = kGroups / kSub;
    constexpr bool kOdd = ROWS == kRowsOne;
    using P = Pair<T>;
    using Raw = typename P::raw;
    extern __shared__ __align__(16) uint8_t smem[];
    float4(*sums)[kGroups][LANES] = reinterpret_cast<float4(*)[kGroups][LANES]>(smem);
    float4(*parts)[8][LANES] = reinterpret_cast<float4(*)[8][LANES]>(sums + 2);
    T* ring = reinterpret_cast<T*>(parts + (CLUSTER ? 2 : 0));
    Mail& mail = *reinterpret_cast<Mail*>(ring + S * kWarps * NT * kPlace);  // (behind the ring; of clusters)
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
    int ta = rank * kTile + warp * kSub * kTok;  // the warp's first token of the tile that is fetched
    int t = rank * kTile + group * kTok;         // this group's first token of the tile that is computed
    W in[NT];
    in[0].start(a.x, b * L, a.x_stride, c0, ta, wl);
    in[1].start(a.r, b * L, a.r_stride, c0, ta, wl);
    in[2].start(a.i, b * L, a.i_stride, c0, ta, wl);
    if (GATED) in[NT - 1].start(a.z, b * L, a.z_stride, c0, ta, wl);
    T* y = static_cast<T*>(a.y) + b * L * a.y_stride + c0;
    const float2 A = load_pair(a.A + c0, lane, have);
    float2 carry = a.init ? load_pair(a.init + b * a.channels + c0, lane, have) : f2(0.f);

    const int64_t strides[5] = {a.x_stride, a.r_stride, a.i_stride, a.z_stride, 0};
    const void* bases[5] = {a.x, a.r, a.i, a.z, nullptr};
    auto ahead = [&](int stage) {
#pragma unroll
        for (int q = 0; q < NT; ++q)
            in[q].fetch(ring + ((stage * kWarps + warp) * NT + q) * kPlace, bases[q], strides[q], ta < n ? ta : -1, n, step, have, wl);
        ta += step;
        commit();
    };
    griddep_launch_dependents();  // (what is launched beside this takes other strips)
    if constexpr (CLUSTER) {
        open_mail(mail);
        cluster_sync();  // the others' shared memory is there
    }
    for (int s = 0; s < S; ++s) ahead(s);
    const int steps = (tiles + K - 1) / K;
    auto walk = [&](auto wide) {
        int stage = 0, buf = 0;
        for (int j = 0; j < steps; ++j, t += step) {
            wait_for<S - 1>();
            __syncwarp();
            const Raw* place = reinterpret_cast<const Raw*>(ring + (stage * kWarps + warp) * NT * kPlace) + wl;
            float2 f[kTok], u[kTok], PA = f2(1.f), PB = f2(0.f);
            Raw z[GATED ? kTok : 1];
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                const float2 x = P::get(place[k * 32]), r = P::get(place[(kTok + k) * 32]),
                             i = P::get(place[(2 * kTok + k) * 32]);
                if (GATED) z[GATED ? k : 0] = place[(3 * kTok + k) * 32];
                float2 m;
                decay2<decltype(wide)::value>(mul2(A, sigmoid2(r)), f[k], m);
                u[k] = mul2(mul2(sqrt2(m), sigmoid2(i)), x);
            }
            if (t + kTok > n) {  // tokens past the row's end leave the state as it is
#pragma unroll
                for (int k = 0; k < kTok; ++k)
                    if (t + k >= n) f[k] = f2(1.f), u[k] = f2(0.f);
            }
#pragma unroll
            for (int k = 0; k < kTok; ++k) PB = fma2(f[k], PB, u[k]), PA = mul2(PA, f[k]);
            sums[buf][group][lane] = make_float4(PA.x, PA.y, PB.x, PB.y);
            __syncthreads();  // (also: the warp's lanes have read their places)
            ahead(stage);
            if (++stage == S) stage = 0;

            // the state that enters the tile, and then this group's tokens
            float2 h = carry, start = carry;
            if constexpr (CLUSTER) {
                PA = f2(1.f), PB = f2(0.f);  // the map of the whole tile
#pragma unroll
                for (int w = 0; w < kGroups; ++w) {
                    const float4 s = sums[buf][w][lane];
                    const float2 sa = make_float2(s.x, s.y);
                    PB = fma2(sa, PB, make_float2(s.z, s.w)), PA = mul2(PA, sa);
                }
                if (group < K) send(&parts[buf][rank][lane], &mail.bars[buf], group, make_float4(PA.x, PA.y, PB.x, PB.y));
                take_mail(mail, j, K * LANES * (int)sizeof(float4), a.status);
                for (int q = 0; q < K; ++q) {
                    if (q == rank) start = carry;
                    const float4 s = parts[buf][q][lane];
                    carry = fma2(make_float2(s.x, s.y), carry, make_float2(s.z, s.w));
                }
                h = start;
                for (int w = 0; w < group; ++w) {
                    const float4 s = sums[buf][w][lane];
                    h = fma2(make_float2(s.x, s.y), h, make_float2(s.z, s.w));
                }
            } else {
#pragma unroll
                for (int w = 0; w < kGroups; ++w) {
                    if (w == group) h = carry;
                    const float4 s = sums[buf][w][lane];
                    carry = fma2(make_float2(s.x, s.y), carry, make_float2(s.z, s.w));
                }
            }
            buf ^= 1;
            if (a.chunk_states && group == 0 && j * K + rank < tiles)
                store<float, true>(a.chunk_states + (b * ((L + kTile - 1) / kTile) + j * K + rank) * a.channels + c0,
                                   start, lane, have);
            Rows1<T, kOdd> out;
            out.start(a.y, b * L, a.y_stride, c0, t, lane, 1);
            auto tokens = [&](auto all) {
#pragma unroll
                for (int k = 0; k < kTok; ++k) {
                    h = fma2(f[k], h, u[k]);
                    float2 o = h;
                    if (GATED) {
                        const float2 g = P::get(z[GATED ? k : 0]);
                        o = mul2(h, mul2(g, sigmoid2(g)));  // (h g could pass the largest number where the gate is shut)
                    }
                    out.template put<decltype(all)::value>(o, lane, have, t + k < n);
                }
            };
            if (t + kTok <= n && have == kStrip) tokens(std::true_type{});
            else tokens(std::false_type{});
        }
    };
    if (__syncthreads_and(A.x >= -1.f && A.y >= -1.f)) walk(std::false_type{});
    else walk(std::true_type{});
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (rank == 0 && group == 0 && a.final_state)
        store<float, true>(a.final_state + b * a.channels + c0, carry, lane, have);
    for (int64_t t = n + rank * kGroups + group; t < L; t += K * kGroups)
        store<T, kOdd>(y + t * a.y_stride, f2(0.f), lane, have);
    if (a.chunk_states) {
        const int64_t nc = (L + kTile - 1) / kTile;
        for (int64_t g = tiles + rank * kGroups + group; g < nc; g += K * kGroups)
            store<float, true>(a.chunk_states + (b * nc + g) * a.channels + c0, carry, lane, have);
    }
    if constexpr (CLUSTER) {
        cluster_sync();  // nobody sends to a block that is gone
        griddep_wait();
    }
}

template <typename T, Rows ROWS, bool GATED>
cudaError_t launch(GlrArgs a, cudaStream_t st) {
    a.status = device_status_word();
    constexpr int LANES = kLanes;
    const int64_t per_row = (a.channels + 2 * LANES - 1) / (2 * LANES);
    return launch_all(k_glr_fwd<T, ROWS, GATED, LANES, false>, k_glr_fwd<T, ROWS, GATED, LANES, true>, a, per_row,
                      kBlocks<T, GATED, LANES>, kGroups * LANES, smem_bytes<T, GATED, LANES>(false),
                      smem_bytes<T, GATED, LANES>(true), st);
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
