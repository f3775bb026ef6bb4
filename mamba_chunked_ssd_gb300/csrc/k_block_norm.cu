// k_block_norm.cu — the norms after and before a block, with its gate and the residual sum:
//
//   p = x or w1 N(x);  p *= SiLU(z);  out = res + scale p;  y = w2 N(out),   N(v) = v / sqrt(mean(v^2) + eps)
//
// Bound by memory: x, z and res are read once, out and y are written once.  A thread has eight
// channels, which it keeps while it walks down the rows, so that the weights stay in its
// registers, where the row stays for both sums; rows of more than 8192 channels are split
// between the blocks of a cluster.  Rows come through shared memory, one ahead.  The two sums a row and 37
// instructions an element bound it next to memory: 32768 x 4096 in bf16, gated, 224 us, 6.0 TB/s; 65536 x 1024 123 us, 5.5;
// 8192 x 4096 with an fp32 residual 75 us, 5.4.  The rings start on a line of 128 bytes: 64 bytes off it 16384 x 8192, gated,
// takes 219 us for 209, 32768 x 2560 149 for 146, but 32768 x 4096 223 for 227 and 32768 x 2048 in fp32 207 for 213.
#include "block_norm.cuh"

namespace m2 {
namespace {

using namespace bnorm;

// Rows under way (32768 x 4096 in bf16, gated: two 226 us, three or four 235; in fp32 two are 196 KB for blocks of
// 1024 threads).
template <typename T>
constexpr int ring_rows() { return 2; }
constexpr int kMost = 1024;  // threads of a block, and of an SM (64 registers each)

// CLUSTER: Q blocks share a row, else Q is 1.
template <typename T, typename R, int GRP, bool GATED, bool CLUSTER>
__global__ void __launch_bounds__(kMost, 1) k_block_norm(const BlockNormArgs a, int Q) {
    constexpr int kRing = ring_rows<T>();
    using InT = RowIn<T, GRP>;
    using InR = RowIn<R, GRP>;
    __shared__ Sums<1> smem;
    int count = 0;
    extern __shared__ __align__(128) uint8_t ring[];
    if (!CLUSTER) Q = 1;
    const int rank = CLUSTER ? (int)glr::cluster_rank() : 0;
    const Share<CLUSTER> by = {Q, rank, a.status};
    const uint32_t rows = (uint32_t)a.rows, walker = blockIdx.x / Q, walkers = gridDim.x / Q;  // (rows < 2^31)
    const int64_t c0 = rank * share_of(a.channels, Q);
    const int n = (int)imin64(a.channels - c0, share_of(a.channels, Q));  // this block's channels
    const int bx = InT::place_bytes(blockDim.x), at_res = GATED ? 2 * bx : bx;
    const int per_row = at_res + (a.res ? InR::place_bytes(blockDim.x) : 0);
    const float inv = 1.f / (float)a.channels;

    float2 w1[4], w2[4], sc[4];
    load_weight<GRP>(a.post_weight ? a.post_weight + c0 : nullptr, n, 1.f, w1);
    load_weight<GRP>(a.scale ? a.scale + c0 : nullptr, n, 1.f, sc);
    load_weight<GRP>(a.pre_weight ? a.pre_weight + c0 : nullptr, n, 1.f, w2);
#pragma unroll
    for (int i = 0; i < 4; ++i) w1[i] = mul2(w1[i], sc[i]);

    InT x, z;
    InR res;
    x.start(a.x, walker, a.x_stride, c0);
    if (GATED) z.start(a.z, walker, a.z_stride, c0);
    if (a.res) res.start(a.res, walker, a.res_stride, c0);
    const int64_t sx = walkers * a.x_stride, sz = walkers * a.z_stride, sr = walkers * a.res_stride;
    uint32_t coming = walker;  // the row that is fetched next
    auto ahead = [&](int stage) {
        if (coming < rows) {
            uint8_t* at = ring + stage * per_row;
            x.fetch(at, n, sx);
            if (GATED) z.fetch(at + bx, n, sz);
            if (a.res) res.fetch(at + at_res, n, sr);
        }
        coming += walkers;
        glr::commit();
    };
    for (int k = 0; k < kRing; ++k) {
        uint8_t* at = ring + k * per_row;
        InT::clear(at, n);
        if (GATED) InT::clear(at + bx, n);
        if (a.res) InR::clear(at + at_res, n);
    }
    if constexpr (CLUSTER) {
        glr::open_mail(smem.mail);
        glr::cluster_sync();  // the others' shared memory is there
    }
    for (int k = 0; k < kRing; ++k) ahead(k);
    RowOut<R, GRP> out;
    RowOut<T, GRP> y;
    out.start(a.out, walker, a.out_stride, c0);
    if (a.pre) y.start(a.y, walker, a.y_stride, c0);
    const int64_t so = walkers * a.out_stride, sy = walkers * a.y_stride;
    int stage = 0;
    for (uint32_t row = walker; row < rows; row += walkers) {
        glr::wait_for<kRing - 1>();
        if (!InT::kOwn) __syncthreads();  // the other threads' copies are there too
        const uint8_t* at = ring + stage * per_row;
        auto first = [&](auto* base, int64_t stride) { return base + row * stride + c0; };
        float2 f[4], g[4], v[4];
        InT::read(at, first(static_cast<const T*>(a.x), a.x_stride), n, f);
        if (GATED) InT::template read<true>(at + bx, first(static_cast<const T*>(a.z), a.z_stride), n, g);
        if (a.res) {
            InR::read(at + at_res, first(static_cast<const R*>(a.res), a.res_stride), n, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f2(0.f);
        }
        if (!InT::kOwn) __syncthreads();  // (the place is read)
        ahead(stage);
        if (++stage == kRing) stage = 0;
        float k1 = 1.f;
        if (a.post) {
            float2 s = f2(0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fma2(f[i], f[i], s);
            float ss[1] = {sum_of(s)};
            group_sums(ss, smem, count, by);
            k1 = rsqrtf(fmaf(ss[0], inv, a.eps));
        }
        float2 s = f2(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 p = mul2(mul2(f[i], f2(k1)), w1[i]);
            if (GATED) p = mul2(mul2(p, g[i]), sigmoid2(g[i]));
            v[i] = add2(v[i], p);
            s = fma2(v[i], v[i], s);  // (0 where there is no channel)
        }
        out.write(n, v, so);
        if (a.pre) {
            float ss[1] = {sum_of(s)};
            group_sums(ss, smem, count, by);
            const float k2 = rsqrtf(fmaf(ss[0], inv, a.eps));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(mul2(v[i], f2(k2)), w2[i]);
            y.write(n, v, sy);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (CLUSTER) glr::cluster_sync();  // nobody sends to a block that is gone
}

template <typename T, typename R, int GRP>
cudaError_t launch_g(BlockNormArgs a, cudaStream_t st) {
    Plan p = plan_of(a.rows, a.channels, kMost);
    if (p.Q > 1) a.status = device_status_word();
    const int bx = RowIn<T, GRP>::place_bytes(p.threads), br = RowIn<R, GRP>::place_bytes(p.threads);
    const int bytes = ring_rows<T>() * (bx * (a.z ? 2 : 1) + (a.res ? br : 0));
    if (p.Q > 1)
        return launch_rows(a.z ? k_block_norm<T, R, GRP, true, true> : k_block_norm<T, R, GRP, false, true>, a, p, a.rows, bytes, st);
    return launch_rows(a.z ? k_block_norm<T, R, GRP, true, false> : k_block_norm<T, R, GRP, false, false>, a, p, a.rows, bytes, st);
}

template <typename T, typename R>
cudaError_t launch_t(const BlockNormArgs& a, cudaStream_t st) {
    const uint64_t t = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.z) |
                       (uint64_t)((a.x_stride | (a.y ? a.y_stride : 0) | (a.z ? a.z_stride : 0)) * sizeof(T));
    const uint64_t r = reinterpret_cast<uintptr_t>(a.res) | reinterpret_cast<uintptr_t>(a.out) |
                       (uint64_t)((a.out_stride | (a.res ? a.res_stride : 0)) * sizeof(R));
    switch (group_of(t, r, a.channels, sizeof(T), sizeof(R))) {
        case 8:
            if constexpr (sizeof(R) == 2) return launch_g<T, R, 8>(a, st);
        case 4: return launch_g<T, R, 4>(a, st);
        case 2: return launch_g<T, R, 2>(a, st);
        default: return launch_g<T, R, 1>(a, st);
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, bool bf16, bool res_bf16, cudaStream_t st) {
    if (!bf16) return launch_t<float, float>(a, st);
    return res_bf16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_t<__nv_bfloat16, float>(a, st);
}

}  // namespace m2
