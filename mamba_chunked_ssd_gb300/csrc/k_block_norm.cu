// k_block_norm.cu — the norms after and before a block, with its gate and the residual sum:
//
//   p = x or w1 N(x);  p *= SiLU(z);  out = res + scale p;  y = w2 N(out),   N(v) = v / sqrt(mean(v^2) + eps)
//
// Bound by memory: x, z and res are read once, out and y are written once.  A thread has eight
// channels, which it keeps while it walks down the rows, so that the weights stay in its
// registers, where the row stays for both sums; rows of more than 4096 channels are split
// between the blocks of a cluster.  Rows come through shared memory, two ahead.
#include "block_norm.cuh"

namespace m2 {
namespace {

using namespace bnorm;

constexpr int kRing = 3;

template <typename T, typename R, int VEC, int TPG>
__global__ void __launch_bounds__(TPG, 1024 / TPG) k_block_norm(const BlockNormArgs a, int Q) {
    constexpr int NV = kPer / VEC;
    constexpr bool kUseRing = VEC > 1;
    using PT = Piece<T, VEC>;
    using PR = Piece<R, VEC>;
    __shared__ Sums<1> smem;
    int turn = 0;
    extern __shared__ __align__(16) uint8_t ring[];
    const int rank = Q > 1 ? (int)glr::cluster_rank() : 0;
    const int64_t walker = blockIdx.x / Q, walkers = gridDim.x / Q;
    const int64_t share = share_of(a.channels, Q), cb = rank * share;  // this block's channels
    const int nvec = (int)((imin64(a.channels - cb, share) + VEC - 1) / VEC);
    const T* x = static_cast<const T*>(a.x) + cb;
    const T* z = a.z ? static_cast<const T*>(a.z) + cb : nullptr;
    const R* res = a.res ? static_cast<const R*>(a.res) + cb : nullptr;
    R* out = static_cast<R*>(a.out) + cb;
    T* y = a.pre ? static_cast<T*>(a.y) + cb : nullptr;
    const float count = (float)a.channels;

    float w1[NV][VEC], w2[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int j = threadIdx.x + i * TPG;
            const int64_t c = cb + (int64_t)j * VEC + e;
            w1[i][e] = (a.post_weight && j < nvec ? a.post_weight[c] : 1.f) * (a.scale && j < nvec ? a.scale[c] : 1.f);
            w2[i][e] = a.pre_weight && j < nvec ? a.pre_weight[c] : 1.f;
        }

    // a thread's places of a stage: its pieces of x, z and res
    auto place = [&](int stage, int i) {
        return ring + (stage * NV + i) * TPG * (int)(2 * sizeof(PT) + sizeof(PR));
    };
    auto ahead = [&](int64_t row, int stage) {
        if constexpr (kUseRing) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = threadIdx.x + i * TPG;
                if (row < a.rows && j < nvec) {
                    const int64_t c = (int64_t)j * VEC;
                    PT* p = reinterpret_cast<PT*>(place(stage, i));
                    copy_piece(p + threadIdx.x, x + row * a.x_stride + c);
                    if (z) copy_piece(p + TPG + threadIdx.x, z + row * a.z_stride + c);
                    if (res) copy_piece(reinterpret_cast<PR*>(p + 2 * TPG) + threadIdx.x, res + row * a.res_stride + c);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    if (Q > 1) glr::cluster_sync();  // the others' shared memory is there
    for (int k = 0; k < kRing; ++k) ahead(walker + k * walkers, k);
    int stage = 0;
    for (int64_t row = walker; row < a.rows; row += walkers) {
        if (kUseRing) asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        PT vx[NV], vz[NV];
        PR vr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = threadIdx.x + i * TPG;
            vx[i] = vz[i] = PT{};
            vr[i] = PR{};
            if (j >= nvec) continue;
            if constexpr (kUseRing) {
                const PT* p = reinterpret_cast<const PT*>(place(stage, i));
                vx[i] = p[threadIdx.x];
                if (z) vz[i] = p[TPG + threadIdx.x];
                if (res) vr[i] = reinterpret_cast<const PR*>(p + 2 * TPG)[threadIdx.x];
            } else {
                const int64_t c = (int64_t)j * VEC;
                load_piece(vx[i], x + row * a.x_stride + c);
                if (z) load_piece(vz[i], z + row * a.z_stride + c);
                if (res) load_piece(vr[i], res + row * a.res_stride + c);
            }
        }
        ahead(row + kRing * walkers, stage);
        if (++stage == kRing) stage = 0;
        float k1 = 1.f;
        if (a.post) {
            float ss[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[VEC];
                widen(vx[i], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss[0] = fmaf(f[e], f[e], ss[0]);
            }
            group_sums<TPG, 1>(ss, smem, turn, Q, rank);
            k1 = rsqrtf(ss[0] / count + a.eps);
        }
        float v[NV][VEC], ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = threadIdx.x + i * TPG;
            float f[VEC], g[VEC];
            widen(vx[i], f), widen(vz[i], g), widen(vr[i], v[i]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float p = f[e] * k1 * w1[i][e];
                if (z) p *= g[e] * sigmoid<T>(g[e]);
                v[i][e] += p;
                ss[0] = fmaf(v[i][e], v[i][e], ss[0]);  // (0 where there is no channel)
            }
            if (j < nvec) store_piece(out + row * a.out_stride + (int64_t)j * VEC, v[i]);
        }
        if (a.pre) {
            group_sums<TPG, 1>(ss, smem, turn, Q, rank);
            const float k2 = rsqrtf(ss[0] / count + a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = threadIdx.x + i * TPG;
                if (j >= nvec) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = v[i][e] * k2 * w2[i][e];
                store_piece(y + row * a.y_stride + (int64_t)j * VEC, o);
            }
        }
    }
    if (kUseRing) asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, typename R, int VEC, int TPG>
cudaError_t launch_n(const BlockNormArgs& a, const Plan& p, cudaStream_t st) {
    const int bytes = VEC > 1 ? kRing * TPG * kPer * (2 * (int)sizeof(T) + (int)sizeof(R)) : 0;
    return launch_rows(k_block_norm<T, R, VEC, TPG>, a, p, TPG, bytes, st);
}

template <typename T, typename R, int VEC>
cudaError_t launch_v(const BlockNormArgs& a, cudaStream_t st) {
    const Plan p = plan_of(a.rows, a.channels, 1024);
    switch (p.threads) {
        case 32: return launch_n<T, R, VEC, 32>(a, p, st);
        case 64: return launch_n<T, R, VEC, 64>(a, p, st);
        case 128: return launch_n<T, R, VEC, 128>(a, p, st);
        case 256: return launch_n<T, R, VEC, 256>(a, p, st);
        default: return launch_n<T, R, VEC, 512>(a, p, st);
    }
}

template <typename T, typename R>
cudaError_t launch_t(const BlockNormArgs& a, cudaStream_t st) {
    const uint64_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                       reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.res) |
                       reinterpret_cast<uintptr_t>(a.out);
    const uint64_t s = (uint64_t)((a.x_stride | (a.y ? a.y_stride : 0) | (a.z ? a.z_stride : 0) | a.channels) * sizeof(T)) |
                       (uint64_t)((a.out_stride | (a.res ? a.res_stride : 0)) * sizeof(R));
    return (p | s) % 16 == 0 ? launch_v<T, R, 16 / sizeof(T)>(a, st) : launch_v<T, R, 1>(a, st);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, bool bf16, bool res_bf16, cudaStream_t st) {
    if (!bf16) return launch_t<float, float>(a, st);
    return res_bf16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_t<__nv_bfloat16, float>(a, st);
}

}  // namespace m2
