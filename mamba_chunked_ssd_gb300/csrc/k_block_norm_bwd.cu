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
// more than 4096 channels are split between the blocks of a cluster, which send one another their sums, twice a row.
// Rows come through shared memory, one or two ahead.  About 55 instructions an element and one block of 512
// threads to an SM, which waits at two barriers a row, bound it next to memory: 32768 x 4096 in bf16, gated, 350 us, 6.1
// TB/s; 8192 x 4096 with an fp32 residual 107 us, 5.6 TB/s; 4096 x 8192 142 us, 3.8 TB/s.  (Two rows at a
// time, for half as many barriers: 581 us, their inputs take the registers; blocks of 256 threads and
// clusters from 2048 channels on 716; rings 48 bytes off a line of 128 429.)
#include "block_norm.cuh"

namespace m2 {
namespace {

using namespace bnorm;

// Rows under way: three, two in fp32 (a ring of 164 KB for blocks of 512 threads).
template <typename T>
constexpr int ring_rows() { return sizeof(T) == 2 ? 3 : 2; }
constexpr int kMost = 512;  // threads of a block, and of an SM (128 registers each)

// CLUSTER: Q blocks share a row, else Q is 1.  FULL: both norms and both gradients of residuals are there.
template <typename T, typename R, int GRP, bool GATED, bool CLUSTER, bool FULL>
__global__ void __launch_bounds__(kMost, 1) k_block_norm_bwd(const BlockNormBwdArgs a, int Q) {
    const bool pre = FULL || a.pre, post = FULL || a.post, dout = FULL || a.dout, has_dres = FULL || a.dres;
    constexpr int kRing = ring_rows<T>();
    __shared__ Sums<3> smem3;
    __shared__ Sums<1> smem1;
    int count3 = 0, count1 = 0;
    extern __shared__ __align__(128) uint8_t ring[];
    if (!CLUSTER) Q = 1;
    const int rank = CLUSTER ? (int)glr::cluster_rank() : 0;
    const Share<CLUSTER> by = {Q, rank, a.status};
    using InT = RowIn<T, GRP>;
    using InR = RowIn<R, GRP>;
    const uint32_t rows = (uint32_t)a.rows, walker = blockIdx.x / Q, walkers = gridDim.x / Q;  // (rows < 2^31)
    const int64_t c0 = rank * share_of(a.channels, Q);
    const int n = (int)imin64(a.channels - c0, share_of(a.channels, Q));  // this block's channels
    // places of a row: x, [z], [dy, r], [dr]
    const int bx = InT::place_bytes(blockDim.x), br = InR::place_bytes(blockDim.x);
    const int at_dy = GATED ? 2 * bx : bx, at_r = at_dy + bx, at_dr = pre ? at_r + br : at_dy;
    const int per_row = at_dr + (dout ? br : 0);
    const float inv = 1.f / (float)a.channels;

    float2 w1[4], w2[4], sc[4], s1[4], s2[4], s3[4];
    load_weight<GRP>(a.post_weight ? a.post_weight + c0 : nullptr, n, 1.f, w1);
    load_weight<GRP>(a.scale ? a.scale + c0 : nullptr, n, 1.f, sc);
    load_weight<GRP>(a.pre_weight ? a.pre_weight + c0 : nullptr, n, 1.f, w2);
#pragma unroll
    for (int i = 0; i < 4; ++i) s1[i] = s2[i] = s3[i] = f2(0.f);

    InT x, z, dy;
    InR r, dr;
    x.start(a.x, walker, a.x_stride, c0);
    if (GATED) z.start(a.z, walker, a.z_stride, c0);
    if (pre) dy.start(a.dy, walker, a.dy_stride, c0), r.start(a.out, walker, a.out_stride, c0);
    if (dout) dr.start(a.dout, walker, a.dout_stride, c0);
    const int64_t sx = walkers * a.x_stride, sz = walkers * a.z_stride, sdy = walkers * a.dy_stride,
                  sr = walkers * a.out_stride, sdr = walkers * a.dout_stride;
    uint32_t coming = walker;  // the row that is fetched next
    auto ahead = [&](int stage) {
        if (coming < rows) {
            uint8_t* at = ring + stage * per_row;
            x.fetch(at, n, sx);
            if (GATED) z.fetch(at + bx, n, sz);
            if (pre) dy.fetch(at + at_dy, n, sdy), r.fetch(at + at_r, n, sr);
            if (dout) dr.fetch(at + at_dr, n, sdr);
        }
        coming += walkers;
        glr::commit();
    };
    for (int k = 0; k < kRing; ++k) {
        uint8_t* at = ring + k * per_row;
        InT::clear(at, n);
        if (GATED) InT::clear(at + bx, n);
        if (pre) InT::clear(at + at_dy, n), InR::clear(at + at_r, n);
        if (dout) InR::clear(at + at_dr, n);
    }
    tc::griddep_launch_dependents();  // the sum over the walkers may be launched; it waits for this grid's end
    if constexpr (CLUSTER) {
        glr::open_mail(smem3.mail), glr::open_mail(smem1.mail);
        glr::cluster_sync();  // the others' shared memory is there
    }
    for (int k = 0; k < kRing; ++k) ahead(k);
    RowOut<T, GRP> dx, dz;
    RowOut<R, GRP> dres;
    dx.start(a.dx, walker, a.dx_stride, c0);
    if (GATED) dz.start(a.dz, walker, a.dz_stride, c0);
    if (has_dres) dres.start(a.dres, walker, a.dres_stride, c0);
    const int64_t tx = walkers * a.dx_stride, tz = walkers * a.dz_stride, tr = walkers * a.dres_stride;
    int stage = 0;
    for (uint32_t row = walker; row < rows; row += walkers) {
        glr::wait_for<kRing - 1>();
        if (!InT::kOwn) __syncthreads();  // the other threads' copies are there too
        const uint8_t* at = ring + stage * per_row;
        auto first = [&](auto* base, int64_t stride) { return base + row * stride + c0; };
        float2 fx[4], fz[4], fd[4], fr[4], D[4];
        InT::read(at, first(static_cast<const T*>(a.x), a.x_stride), n, fx);
        if (GATED) InT::read(at + bx, first(static_cast<const T*>(a.z), a.z_stride), n, fz);
        if (pre) {
            InT::read(at + at_dy, first(static_cast<const T*>(a.dy), a.dy_stride), n, fd);
            InR::read(at + at_r, first(static_cast<const R*>(a.out), a.out_stride), n, fr);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) fd[i] = fr[i] = f2(0.f);
        }
        if (dout) {
            InR::read(at + at_dr, first(static_cast<const R*>(a.dout), a.dout_stride), n, D);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) D[i] = f2(0.f);
        }
        if (!InT::kOwn) __syncthreads();  // (the place is read)
        ahead(stage);
        if (++stage == kRing) stage = 0;
        float k1 = 1.f, k2 = 0.f, m2 = 0.f;
        if (post || pre) {
            float2 s[3] = {f2(0.f), f2(0.f), f2(0.f)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[0] = fma2(fx[i], fx[i], s[0]);
                s[1] = fma2(fr[i], fr[i], s[1]);
                s[2] = fma2(mul2(fd[i], w2[i]), fr[i], s[2]);
            }
            float sums[3] = {sum_of(s[0]), sum_of(s[1]), sum_of(s[2])};
            group_sums(sums, smem3, count3, by);
            if (post) k1 = rsqrtf(fmaf(sums[0], inv, a.eps));
            if (pre) k2 = rsqrtf(fmaf(sums[1], inv, a.eps));
            m2 = -k2 * k2 * (k2 > 0.f ? sums[2] * inv : 0.f);  // (a sum that k2 = 0 comes from takes this one along)
        }
        float2 last = f2(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s3[i] = fma2(mul2(fd[i], f2(k2)), fr[i], s3[i]);
            D[i] = fma2(f2(k2), fma2(f2(m2), fr[i], mul2(fd[i], w2[i])), D[i]);
            fx[i] = mul2(fx[i], f2(k1));
            float2 v = mul2(fx[i], w1[i]), dn = mul2(D[i], sc[i]);
            if (GATED) {
                const float2 sg = sigmoid2(fz[i]), g = mul2(fz[i], sg);
                fz[i] = mul2(mul2(dn, v), fma2(g, fma2(sg, f2(-1.f), f2(1.f)), sg));  // dz
                v = mul2(v, g), dn = mul2(dn, g);
            }
            s2[i] = fma2(D[i], v, s2[i]);
            s1[i] = fma2(dn, fx[i], s1[i]);
            fd[i] = mul2(dn, w1[i]);
            last = fma2(fd[i], fx[i], last);
        }
        if (has_dres) dres.write(n, D, tr);
        if (GATED) dz.write(n, fz, tz);
        float m1 = 0.f;
        if (post) {
            float sums[1] = {sum_of(last)};
            group_sums(sums, smem1, count1, by);
            m1 = -sums[0] * inv;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) fd[i] = mul2(f2(k1), fma2(f2(m1), fx[i], fd[i]));
        dx.write(n, fd, tx);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float* part = a.partials + (int64_t)walker * 3 * a.channels + c0;
    store_weight<GRP>(part, n, s1);
    store_weight<GRP>(part + a.channels, n, s2);
    store_weight<GRP>(part + 2 * a.channels, n, s3);
    if constexpr (CLUSTER) glr::cluster_sync();  // nobody sends to a block that is gone
}

// (In bf16, 32768 x 4096, gated: 351 us, without it 390; narrow groups are bound by their loads.)
template <typename T, typename R, int GRP, bool CLUSTER>
auto pick(const BlockNormBwdArgs& a) {
    if constexpr (GRP >= 4)
        if (a.pre && a.post && a.dout && a.dres)
            return a.z ? k_block_norm_bwd<T, R, GRP, true, CLUSTER, true> : k_block_norm_bwd<T, R, GRP, false, CLUSTER, true>;
    return a.z ? k_block_norm_bwd<T, R, GRP, true, CLUSTER, false> : k_block_norm_bwd<T, R, GRP, false, CLUSTER, false>;
}

template <typename T, typename R, int GRP>
cudaError_t launch_g(BlockNormBwdArgs a, cudaStream_t st) {
    Plan p = plan_of(a.rows, a.channels, kMost);
    if (p.Q > 1) a.status = device_status_word();
    const int bx = RowIn<T, GRP>::place_bytes(p.threads), br = RowIn<R, GRP>::place_bytes(p.threads);
    const int bytes = ring_rows<T>() * (bx * (1 + (a.z != nullptr) + a.pre) + br * (a.pre + (a.dout != nullptr)));
    const cudaError_t e = launch_rows(p.Q > 1 ? pick<T, R, GRP, true>(a) : pick<T, R, GRP, false>(a), a, p, a.rows, bytes, st);
    if (e != cudaSuccess || (!a.dpost && !a.dscale && !a.dpre)) return e;
    return launch_sum_rows(a.partials, p.walkers, {a.dpost, a.channels}, {a.dscale, a.channels}, {a.dpre, a.channels},
                           nullptr, st);
}

template <typename T, typename R>
cudaError_t launch_t(const BlockNormBwdArgs& a, cudaStream_t st) {
    uint64_t t = 0, r = 0;
    for (const void* p : {a.x, a.z, a.dy, (const void*)a.dx, (const void*)a.dz}) t |= reinterpret_cast<uintptr_t>(p);
    for (const void* p : {a.out, a.dout, (const void*)a.dres}) r |= reinterpret_cast<uintptr_t>(p);
    t |= (uint64_t)((a.x_stride | a.dx_stride | (a.z ? a.z_stride | a.dz_stride : 0) | (a.dy ? a.dy_stride : 0)) * sizeof(T));
    r |= (uint64_t)(((a.out ? a.out_stride : 0) | (a.dout ? a.dout_stride : 0) | (a.dres ? a.dres_stride : 0)) * sizeof(R));
    switch (group_of(t, r, a.channels, sizeof(T), sizeof(R))) {
        case 8:
            if constexpr (sizeof(R) == 2) return launch_g<T, R, 8>(a, st);
        case 4: return launch_g<T, R, 4>(a, st);
        case 2: return launch_g<T, R, 2>(a, st);
        default: return launch_g<T, R, 1>(a, st);
    }
}

}  // namespace

int64_t block_norm_bwd_partials(int64_t rows, int64_t channels) {
    return plan_of(rows, channels, kMost).walkers * 3 * channels;
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, bool bf16, bool res_bf16, cudaStream_t st) {
    if (!bf16) return launch_t<float, float>(a, st);
    return res_bf16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_t<__nv_bfloat16, float>(a, st);
}

}  // namespace m2
