// k_gdr_step.cu — the gated delta rule's one-token step (decoding).
//
//   h <- a h + k (beta (v - a h^T k))^T,  y = scale h^T q,   a = e^g
//
// The state is read and written once, 8 S H bytes per (batch row, head), next
// to a few hundred bytes of q, k, v: the step is bound by memory.  A block owns
// 16 to 64 columns of one head's state (columns do not meet) and keeps them in
// registers, read before anything they wait for.  The two column sums r = h^T k
// and p = h^T q are formed together over the state that was read, so the block
// meets once: with r and p,
//   w = beta (v - a r),   y = scale (a p + (q . k) w),   h <- a h + k w^T.
// 256 sequences of 64 heads of 64 columns, S 128: 158 us, 6.9 TB/s (1.02 of a plain
// copy; 155 where the blocks' widths below were compared).
#include "gated_delta.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 128;

// VEC columns per thread (4, or 1 where H is no multiple of 4), RPT state rows
// per thread; COLS / VEC threads span the columns, kRows row groups the rows.
template <typename T, int COLS, int VEC, int RPT>
__global__ void __launch_bounds__(kThreads) k_gdr_step(const GdrArgs a) {
    constexpr int kCt = COLS / VEC, kRows = kThreads / kCt;
    using V = typename VecOf<float, VEC>::type;
    __shared__ float s_q[256], s_k[256], s_red[4][3], s_part[4][COLS][2];
    const Geom& g = a.g;
    const int S = (int)g.dstate, H = (int)g.headdim;
    const int64_t h = blockIdx.y, b = blockIdx.z;
    const int64_t grp = h / g.heads_per_group;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ct = tid % kCt, r0 = tid / kCt;
    const int col = blockIdx.x * COLS + ct * VEC;
    const bool live = col < H;
    const int64_t base = (b * g.nheads + h) * (int64_t)S * H + col;

    float hv[RPT][VEC];
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int s = r0 + u * kRows;
        V t = V{};
        if (live && a.init && s < S) t = *reinterpret_cast<const V*>(a.init + base + (int64_t)s * H);
        unpack<VEC>(t, hv[u], (const float*)nullptr);
    }

    const T* q = static_cast<const T*>(a.q) + b * a.q_stride + grp * S;
    const T* k = static_cast<const T*>(a.k) + b * a.k_stride + grp * S;
    float qq = 0.f, kk = 0.f, qk = 0.f;
    for (int i = tid; i < kRows * RPT; i += kThreads) {  // zeros past S: rows that no state has
        const float fq = i < S ? to_f32(q[i]) : 0.f, fk = i < S ? to_f32(k[i]) : 0.f;
        s_q[i] = fq;
        s_k[i] = fk;
        qq = fmaf(fq, fq, qq);
        kk = fmaf(fk, fk, kk);
        qk = fmaf(fq, fk, qk);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        qq += __shfl_xor_sync(0xffffffffu, qq, m);
        kk += __shfl_xor_sync(0xffffffffu, kk, m);
        qk += __shfl_xor_sync(0xffffffffu, qk, m);
    }
    if (lane == 0) s_red[warp][0] = qq, s_red[warp][1] = kk, s_red[warp][2] = qk;
    __syncthreads();

    float r[VEC], p[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) r[e] = p[e] = 0.f;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const float fk = s_k[r0 + u * kRows], fq = s_q[r0 + u * kRows];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            r[e] = fmaf(fk, hv[u][e], r[e]);
            p[e] = fmaf(fq, hv[u][e], p[e]);
        }
    }
    // a column's rows: over the lanes of a warp that share it, then over the warps
#pragma unroll
    for (int m = kCt; m < 32; m <<= 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            r[e] += __shfl_xor_sync(0xffffffffu, r[e], m);
            p[e] += __shfl_xor_sync(0xffffffffu, p[e], m);
        }
    }
    if (lane < kCt) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s_part[warp][ct * VEC + e][0] = r[e], s_part[warp][ct * VEC + e][1] = p[e];
    }
    __syncthreads();
    if (!live) return;

    const int64_t bh = b * g.nheads + h;
    const float dec = expf(a.gate[bh]), beta = a.beta[bh];
    qq = s_red[0][0] + s_red[1][0] + s_red[2][0] + s_red[3][0];
    kk = s_red[0][1] + s_red[1][1] + s_red[2][1] + s_red[3][1];
    qk = s_red[0][2] + s_red[1][2] + s_red[2][2] + s_red[3][2];
    const float nq = a.l2norm ? rsqrtf(qq + a.l2_eps) : 1.f, nk = a.l2norm ? rsqrtf(kk + a.l2_eps) : 1.f;
    const T* v = static_cast<const T*>(a.v) + b * a.v_stride + h * H + col;
    float w[VEC], o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const int c = ct * VEC + e;
        const float rc = s_part[0][c][0] + s_part[1][c][0] + s_part[2][c][0] + s_part[3][c][0];
        const float pc = s_part[0][c][1] + s_part[1][c][1] + s_part[2][c][1] + s_part[3][c][1];
        const float vc = to_f32(v[e]);
        const float wc = beta * fmaf(-dec, nk * rc, vc);
        o[e] = a.scale * nq * fmaf(dec, pc, nk * qk * wc);
        w[e] = nk * wc;
    }
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
        const int s = r0 + u * kRows;
        if (s >= S) break;
        const float fk = s_k[s];
#pragma unroll
        for (int e = 0; e < VEC; ++e) hv[u][e] = fmaf(fk, w[e], dec * hv[u][e]);
        *reinterpret_cast<V*>(a.final_state + base + (int64_t)s * H) = pack<float, VEC>(hv[u]);
    }
    if (r0 == 0) {
        T* y = static_cast<T*>(a.y) + bh * H + col;
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = from_f32<T>(o[e]);
    }
}

template <typename T, int COLS, int VEC>
cudaError_t launch_c(const GdrArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.g.headdim + COLS - 1) / COLS), (unsigned)a.g.nheads, (unsigned)a.g.batch);
    constexpr int kRows = kThreads / (COLS / VEC);
    const int64_t S = a.g.dstate;
    if (S <= 64)
        k_gdr_step<T, COLS, VEC, 64 / kRows><<<grid, kThreads, 0, st>>>(a);
    else if (S <= 128)
        k_gdr_step<T, COLS, VEC, 128 / kRows><<<grid, kThreads, 0, st>>>(a);
    else
        k_gdr_step<T, COLS, VEC, 256 / kRows><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

// Columns per block: 64 where that still gives eight blocks to an SM (more bytes under way
// for each meeting of a block), 16 for narrow heads, else 32.  us with 16 / 32 / 64: 256
// sequences of 64 heads of 64, S 128, 186 / 165 / 155; of 40, S 64, 100 / 79 / 71; of 8, S 128,
// 40 / 55 / 87; one sequence of 32 heads of 128, S 128, 3.3 / 3.1 / 3.7.
template <typename T>
cudaError_t launch_t(const GdrArgs& a, cudaStream_t st) {
    const int64_t H = a.g.headdim;
    if (H % 4 != 0) return launch_c<T, 32, 1>(a, st);
    if (H <= 16) return launch_c<T, 16, 4>(a, st);
    const int sms = sm_count();
    const bool many = a.g.batch * a.g.nheads * ((H + 63) / 64) >= 8 * (int64_t)(sms > 0 ? sms : 152);
    return H > 32 && many ? launch_c<T, 64, 4>(a, st) : launch_c<T, 32, 4>(a, st);
}

}  // namespace

cudaError_t launch_gdr_step(const GdrArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
