// k_block_norm_bwd.cu — gradients of the block norm.  With k1, k2 the factors 1 / sqrt(mean(v^2) + eps) of
// x and of the sum r that the forward pass wrote, n = w1 k1 x, g = SiLU(z):
//
//   D  = dr + k2 (w2 dy - r k2^2 mean(w2 dy r))     dres = D,  dw2 = sum_rows dy k2 r
//   dp = scale D                                    dscale = sum_rows D n g
//   dz = dp n SiLU'(z),  q = dp g                   dw1 = sum_rows q k1 x
//   dx = k1 (w1 q - k1 x mean(w1 q k1 x))
//
// Bound by memory: every row is read once and written once, its factors are computed again.
// Two sums over a row's threads: x^2, r^2 and w2 dy r together, then w1 q k1 x.
// A thread has eight channels, which it keeps while it walks down the rows: weights, and the sums
// over the rows, stay in its registers; the sums of all walkers are added up by a second kernel.  Rows of
// more than 4096 channels are split between the blocks of a cluster.  Rows come through
// shared memory, one or two ahead.
#include "block_norm.cuh"

namespace m2 {
namespace {

using namespace bnorm;

// Rows under way: three, two in fp32 (a ring of 164 KB for blocks of 512 threads).
template <typename T>
constexpr int ring_rows() { return sizeof(T) == 2 ? 3 : 2; }
constexpr int kResident = 512;  // threads of an SM at once
// Bytes of a thread's places in the ring, a row.
template <typename T, typename R>
constexpr int place_bytes() {
    return kPer * (3 * (int)sizeof(T) + 2 * (int)sizeof(R));
}

template <typename T, typename R, int VEC, int TPG>
__global__ void __launch_bounds__(TPG, kResident / TPG) k_block_norm_bwd(const BlockNormBwdArgs a, int Q) {
    constexpr int NV = kPer / VEC, kRing = ring_rows<T>();
    constexpr bool kUseRing = VEC > 1;
    __shared__ Sums<3> smem3;
    __shared__ Sums<1> smem1;
    int turn3 = 0, turn1 = 0;
    extern __shared__ __align__(16) uint8_t ring[];
    const int rank = Q > 1 ? (int)glr::cluster_rank() : 0;
    const int64_t walker = blockIdx.x / Q, walkers = gridDim.x / Q;
    const int64_t share = share_of(a.channels, Q), cb = rank * share;  // this block's channels
    const int nvec = (int)((imin64(a.channels - cb, share) + VEC - 1) / VEC);
    const T* x = static_cast<const T*>(a.x) + cb;
    const T* z = a.z ? static_cast<const T*>(a.z) + cb : nullptr;
    const T* dy = a.pre ? static_cast<const T*>(a.dy) + cb : nullptr;
    const R* r = a.pre ? static_cast<const R*>(a.out) + cb : nullptr;
    const R* dr = a.dout ? static_cast<const R*>(a.dout) + cb : nullptr;
    T* dx = static_cast<T*>(a.dx) + cb;
    T* dz = a.z ? static_cast<T*>(a.dz) + cb : nullptr;
    R* dres = a.dres ? static_cast<R*>(a.dres) + cb : nullptr;
    const float count = (float)a.channels;

    float w1[NV][VEC], w2[NV][VEC], sc[NV][VEC], s1[NV][VEC], s2[NV][VEC], s3[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int j = threadIdx.x + i * TPG;
            const int64_t c = cb + (int64_t)j * VEC + e;
            w1[i][e] = a.post_weight && j < nvec ? a.post_weight[c] : 1.f;
            w2[i][e] = a.pre_weight && j < nvec ? a.pre_weight[c] : 1.f;
            sc[i][e] = a.scale && j < nvec ? a.scale[c] : 1.f;
            s1[i][e] = s2[i][e] = s3[i][e] = 0.f;
        }

    struct Row {
        Piece<T, VEC> x, z, dy;
        Piece<R, VEC> r, dr;
    };
    auto ahead = [&](int64_t row, int stage) {
        if constexpr (kUseRing) {
            uint8_t* at = ring + stage * TPG * NV * (int)sizeof(Row);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = threadIdx.x + i * TPG;
                if (row < a.rows && j < nvec) {
                    const int64_t c = (int64_t)j * VEC;
                    auto to = [&](auto* p, int before) {
                        return reinterpret_cast<decltype(p)>(at + before * TPG * NV) + i * TPG + threadIdx.x;
                    };
                    constexpr int t = sizeof(Piece<T, VEC>), u = sizeof(Piece<R, VEC>);
                    copy_piece(to((Piece<T, VEC>*)nullptr, 0), x + row * a.x_stride + c);
                    if (z) copy_piece(to((Piece<T, VEC>*)nullptr, t), z + row * a.z_stride + c);
                    if (dy) copy_piece(to((Piece<T, VEC>*)nullptr, 2 * t), dy + row * a.dy_stride + c);
                    if (r) copy_piece(to((Piece<R, VEC>*)nullptr, 3 * t), r + row * a.out_stride + c);
                    if (dr) copy_piece(to((Piece<R, VEC>*)nullptr, 3 * t + u), dr + row * a.dout_stride + c);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto take = [&](Row& v, int64_t row, int stage, int i) {
        const int j = threadIdx.x + i * TPG;
        v = Row{};
        if (j >= nvec) return;
        if constexpr (kUseRing) {
            const uint8_t* at = ring + stage * TPG * NV * (int)sizeof(Row);
            auto from = [&](auto* p, int before) {
                return reinterpret_cast<decltype(p)>(at + before * TPG * NV) + i * TPG + threadIdx.x;
            };
            constexpr int t = sizeof(Piece<T, VEC>), u = sizeof(Piece<R, VEC>);
            v.x = *from((const Piece<T, VEC>*)nullptr, 0);
            if (z) v.z = *from((const Piece<T, VEC>*)nullptr, t);
            if (dy) v.dy = *from((const Piece<T, VEC>*)nullptr, 2 * t);
            if (r) v.r = *from((const Piece<R, VEC>*)nullptr, 3 * t);
            if (dr) v.dr = *from((const Piece<R, VEC>*)nullptr, 3 * t + u);
        } else {
            const int64_t c = (int64_t)j * VEC;
            load_piece(v.x, x + row * a.x_stride + c);
            if (z) load_piece(v.z, z + row * a.z_stride + c);
            if (dy) load_piece(v.dy, dy + row * a.dy_stride + c);
            if (r) load_piece(v.r, r + row * a.out_stride + c);
            if (dr) load_piece(v.dr, dr + row * a.dout_stride + c);
        }
    };
    if (Q > 1) glr::cluster_sync();  // the others' shared memory is there
    for (int k = 0; k < kRing; ++k) ahead(walker + k * walkers, k);
    int stage = 0;
    for (int64_t row = walker; row < a.rows; row += walkers) {
        if (kUseRing) asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        Row v[NV];
        float sums[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            take(v[i], row, stage, i);
            float fx[VEC], fr[VEC], fd[VEC];
            widen(v[i].x, fx), widen(v[i].r, fr), widen(v[i].dy, fd);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                sums[0] = fmaf(fx[e], fx[e], sums[0]);
                sums[1] = fmaf(fr[e], fr[e], sums[1]);
                sums[2] = fmaf(fd[e] * w2[i][e], fr[e], sums[2]);
            }
        }
        ahead(row + kRing * walkers, stage);
        if (++stage == kRing) stage = 0;
        group_sums<TPG, 3>(sums, smem3, turn3, Q, rank);
        const float k1 = a.post ? rsqrtf(sums[0] / count + a.eps) : 1.f;
        const float k2 = a.pre ? rsqrtf(sums[1] / count + a.eps) : 0.f;
        const float m2 = k2 * k2 * (sums[2] / count);
        float q[NV][VEC], last[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = threadIdx.x + i * TPG;
            const int64_t c = (int64_t)j * VEC;
            float fx[VEC], fz[VEC], fr[VEC], fd[VEC], D[VEC], oz[VEC];
            widen(v[i].x, fx), widen(v[i].z, fz), widen(v[i].r, fr), widen(v[i].dy, fd), widen(v[i].dr, D);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s3[i][e] = fmaf(fd[e] * k2, fr[e], s3[i][e]);
                D[e] = fmaf(k2, fmaf(-m2, fr[e], fd[e] * w2[i][e]), D[e]);
                const float xh = fx[e] * k1, n = xh * w1[i][e];
                float g = 1.f, dn = D[e] * sc[i][e];
                if (z) {
                    const float sg = sigmoid<T>(fz[e]);
                    g = fz[e] * sg;
                    oz[e] = dn * n * fmaf(g, 1.f - sg, sg);
                }
                s2[i][e] = fmaf(D[e], n * g, s2[i][e]);
                dn *= g;
                s1[i][e] = fmaf(dn, xh, s1[i][e]);
                q[i][e] = dn * w1[i][e];
                last[0] = fmaf(q[i][e], xh, last[0]);
            }
            if (j < nvec) {
                if (dres) store_piece(dres + row * a.dres_stride + c, D);
                if (z) store_piece(dz + row * a.dz_stride + c, oz);
            }
        }
        float m1 = 0.f;
        if (a.post) {
            group_sums<TPG, 1>(last, smem1, turn1, Q, rank);
            m1 = k1 * (last[0] / count);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = threadIdx.x + i * TPG;
            if (j >= nvec) continue;
            float fx[VEC], o[VEC];
            widen(v[i].x, fx);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = k1 * fmaf(-m1, fx[e], q[i][e]);
            store_piece(dx + row * a.dx_stride + (int64_t)j * VEC, o);
        }
    }
    if (kUseRing) asm volatile("cp.async.wait_all;" ::: "memory");
    float* part = a.partials + walker * 3 * a.channels + cb;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = threadIdx.x + i * TPG;
        if (j >= nvec) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int64_t c = (int64_t)j * VEC + e;
            part[c] = s1[i][e], part[a.channels + c] = s2[i][e], part[2 * a.channels + c] = s3[i][e];
        }
    }
}

template <typename T, typename R, int VEC, int TPG>
cudaError_t launch_n(const BlockNormBwdArgs& a, const Plan& p, cudaStream_t st) {
    const int bytes = VEC > 1 ? ring_rows<T>() * TPG * place_bytes<T, R>() : 0;
    const cudaError_t e = launch_rows(k_block_norm_bwd<T, R, VEC, TPG>, a, p, TPG, bytes, st);
    if (e != cudaSuccess) return e;
    if (!a.dpost && !a.dscale && !a.dpre) return cudaSuccess;
    return launch_sum_rows(a.partials, p.walkers, {a.dpost, a.channels}, {a.dscale, a.channels}, {a.dpre, a.channels},
                           nullptr, st);
}

template <typename T, typename R, int VEC>
cudaError_t launch_v(const BlockNormBwdArgs& a, cudaStream_t st) {
    const Plan p = plan_of(a.rows, a.channels, kResident);
    switch (p.threads) {
        case 32: return launch_n<T, R, VEC, 32>(a, p, st);
        case 64: return launch_n<T, R, VEC, 64>(a, p, st);
        case 128: return launch_n<T, R, VEC, 128>(a, p, st);
        case 256: return launch_n<T, R, VEC, 256>(a, p, st);
        default: return launch_n<T, R, VEC, 512>(a, p, st);
    }
}

template <typename T, typename R>
cudaError_t launch_t(const BlockNormBwdArgs& a, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const void* ptr[] = {a.x, a.z, a.dy, a.dx, a.dz, a.out, a.dout, a.dres};
    uint64_t all = (uint64_t)a.channels * sizeof(T);
    for (const void* p : ptr) all |= reinterpret_cast<uintptr_t>(p);
    all |= (uint64_t)((a.x_stride | a.dx_stride | (a.z ? a.z_stride | a.dz_stride : 0) | (a.dy ? a.dy_stride : 0)) * sizeof(T));
    all |= (uint64_t)(((a.out ? a.out_stride : 0) | (a.dout ? a.dout_stride : 0) | (a.dres ? a.dres_stride : 0)) * sizeof(R));
    if (all % 16 == 0) return launch_v<T, R, VEC>(a, st);
    return launch_v<T, R, 1>(a, st);
}

}  // namespace

int64_t block_norm_bwd_partials(int64_t rows, int64_t channels) {
    return plan_of(rows, channels, kResident).walkers * 3 * channels;
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool bf16, bool res_bf16, cudaStream_t st) {
    if (!bf16) return launch_t<float, float>(a, st);
    return res_bf16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_t<__nv_bfloat16, float>(a, st);
}

}  // namespace m2
