// k_gdr_recurrent.cu — the gated delta rule token by token on the CUDA cores,
// for every shape and dtype:
//
//   h <- a h + k (beta (v - a h^T k))^T,  y = scale h^T q,   a = e^g
//
// Columns of the state do not meet, so a block owns 16 columns of one head for
// the whole sequence, four to a warp, and a column's rows lie in the registers
// of eight lanes.  What bounds it is the chain from one token's state to the
// next one's: the sum h^T k over the rows (registers, then three shuffles), the
// correction, the update.  The outputs are kept off that chain: p = h^T q is
// summed beside r = h^T k over the state before the update, and
//   w = beta (v - a r),   y = scale (a p + (q . k) w),   h <- a h + k w^T.
// Sixteen tokens at a time are staged in shared memory as fp32, normalised
// there where asked, while the next sixteen are on their way in registers; a
// token's row is read from there while the token before is computed.
#include "gated_delta.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 16;   // columns per block
constexpr int kTok = 16;    // tokens per tile: eight threads stage each token's row

// RP: state rows per lane (8 lanes span S <= 8 RP rows).
template <typename T, int RP>
__global__ void __launch_bounds__(kThreads) k_gdr_recurrent(const GdrArgs a) {
    constexpr int kS = 8 * RP;
    __shared__ __align__(16) float s_k[kTok][kS], s_q[kTok][kS];
    __shared__ float s_v[kTok][kCols], s_y[kTok][kCols];
    __shared__ float4 s_c[kTok];  // decay, beta, scale of the output, q . k
    const Geom& g = a.g;
    const int S = (int)g.dstate, H = (int)g.headdim;
    const int64_t h = blockIdx.y, b = blockIdx.z;
    const int64_t L = g.seqlen, n = row_length(a.lengths, b, L);
    const int64_t grp = h / g.heads_per_group;
    const int tid = threadIdx.x;
    const int row = tid / 8, part = tid % 8;          // staging: token row, eighth of the row
    const int c = (tid / 32) * 4 + (tid % 32) / 8;    // recurrence: column of the block
    const int rl = tid % 8;                           // rows 32 i + 4 rl + j
    const int col0 = blockIdx.x * kCols;
    const int64_t bh = b * g.nheads + h;

    float hs[RP];
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int s = (i / 4) * 32 + rl * 4 + i % 4;
        hs[i] = (a.init && s < S && col0 + c < H) ? a.init[(bh * S + s) * H + col0 + c] : 0.f;
    }

    const T* q = static_cast<const T*>(a.q) + b * L * a.q_stride + grp * S;
    const T* k = static_cast<const T*>(a.k) + b * L * a.k_stride + grp * S;
    const T* v = static_cast<const T*>(a.v) + b * L * a.v_stride + h * H + col0;
    T* y = static_cast<T*>(a.y) + (b * L * g.nheads + h) * H + col0;

    float kr[RP], qr[RP], vr[2], gr, br;
    auto fetch = [&](int64_t t0) {
        const int64_t t = t0 + row;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const int s = (i / 4) * 32 + part * 4 + i % 4;
            const bool in = t < n && s < S;
            kr[i] = in ? to_f32(k[t * a.k_stride + s]) : 0.f;
            qr[i] = in ? to_f32(q[t * a.q_stride + s]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int cc = part * 2 + i;
            vr[i] = (t < n && col0 + cc < H) ? to_f32(v[t * a.v_stride + cc]) : 0.f;
        }
        gr = t < n ? a.gate[(b * L + t) * g.nheads + h] : 0.f;
        br = t < n ? a.beta[(b * L + t) * g.nheads + h] : 0.f;
    };

    if (n > 0) fetch(0);
    for (int64_t t0 = 0; t0 < n; t0 += kTok) {
        float kk = 0.f, qq = 0.f, qk = 0.f;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            kk = fmaf(kr[i], kr[i], kk);
            qq = fmaf(qr[i], qr[i], qq);
            qk = fmaf(qr[i], kr[i], qk);
        }
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, m);
            qq += __shfl_xor_sync(0xffffffffu, qq, m);
            qk += __shfl_xor_sync(0xffffffffu, qk, m);
        }
        const float nk = a.l2norm ? rsqrtf(kk + a.l2_eps) : 1.f, nq = a.l2norm ? rsqrtf(qq + a.l2_eps) : 1.f;
        __syncthreads();  // the previous tile has been used, its outputs written
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const int s = (i / 4) * 32 + part * 4 + i % 4;
            s_k[row][s] = nk * kr[i];
            s_q[row][s] = qr[i];
        }
        s_v[row][part * 2] = vr[0];
        s_v[row][part * 2 + 1] = vr[1];
        if (part == 0) s_c[row] = make_float4(exp2f(kLog2e * gr), br, a.scale * nq, qk * nk);
        __syncthreads();
        if (t0 + kTok < n) fetch(t0 + kTok);
        const int nt = (int)imin64(kTok, n - t0);
        float4 k4[2][RP / 4], q4[2][RP / 4], co[2];
        float vt[2];
        auto read = [&](int t, int x) {
            co[x] = s_c[t];
            vt[x] = s_v[t][c];
#pragma unroll
            for (int i = 0; i < RP / 4; ++i) {
                k4[x][i] = *reinterpret_cast<const float4*>(&s_k[t][i * 32 + rl * 4]);
                q4[x][i] = *reinterpret_cast<const float4*>(&s_q[t][i * 32 + rl * 4]);
            }
        };
        auto token = [&](int t, int x) {
            float r[4] = {0.f, 0.f, 0.f, 0.f}, p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < RP / 4; ++i) {
                r[0] = fmaf(k4[x][i].x, hs[4 * i], r[0]);
                r[1] = fmaf(k4[x][i].y, hs[4 * i + 1], r[1]);
                r[2] = fmaf(k4[x][i].z, hs[4 * i + 2], r[2]);
                r[3] = fmaf(k4[x][i].w, hs[4 * i + 3], r[3]);
            }
#pragma unroll
            for (int i = 0; i < RP / 4; ++i) {
                p[0] = fmaf(q4[x][i].x, hs[4 * i], p[0]);
                p[1] = fmaf(q4[x][i].y, hs[4 * i + 1], p[1]);
                p[2] = fmaf(q4[x][i].z, hs[4 * i + 2], p[2]);
                p[3] = fmaf(q4[x][i].w, hs[4 * i + 3], p[3]);
            }
            float rs = (r[0] + r[1]) + (r[2] + r[3]), ps = (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
            for (int m = 4; m > 0; m >>= 1) {
                rs += __shfl_xor_sync(0xffffffffu, rs, m);
                ps += __shfl_xor_sync(0xffffffffu, ps, m);
            }
            const float w = co[x].y * fmaf(-co[x].x, rs, vt[x]);
#pragma unroll
            for (int i = 0; i < RP / 4; ++i) {
                hs[4 * i] = fmaf(k4[x][i].x, w, co[x].x * hs[4 * i]);
                hs[4 * i + 1] = fmaf(k4[x][i].y, w, co[x].x * hs[4 * i + 1]);
                hs[4 * i + 2] = fmaf(k4[x][i].z, w, co[x].x * hs[4 * i + 2]);
                hs[4 * i + 3] = fmaf(k4[x][i].w, w, co[x].x * hs[4 * i + 3]);
            }
            if (rl == 0) s_y[t][c] = co[x].z * fmaf(co[x].x, ps, co[x].w * w);
        };
        read(0, 0);
        for (int t = 0; t < nt; t += 2) {  // (rows past nt are zeros, and stay unused)
            read(t + 1, 1);
            token(t, 0);
            if (t + 1 >= nt) break;
            read(t + 2 < kTok ? t + 2 : 0, 0);
            token(t + 1, 1);
        }
        __syncthreads();
        if (row < nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int cc = part * 2 + i;
                if (col0 + cc < H) y[(t0 + row) * g.nheads * H + cc] = from_f32<T>(s_y[row][cc]);
            }
        }
    }
    for (int64_t t = n + row; t < L; t += kTok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int cc = part * 2 + i;
            if (col0 + cc < H) y[t * g.nheads * H + cc] = from_f32<T>(0.f);
        }
    }
    if (a.final_state && col0 + c < H) {
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const int s = (i / 4) * 32 + rl * 4 + i % 4;
            if (s < S) a.final_state[(bh * S + s) * H + col0 + c] = hs[i];
        }
    }
}

template <typename T>
cudaError_t launch_t(const GdrArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.g.headdim + kCols - 1) / kCols), (unsigned)a.g.nheads, (unsigned)a.g.batch);
    if (a.g.dstate <= 64)
        k_gdr_recurrent<T, 8><<<grid, kThreads, 0, st>>>(a);
    else if (a.g.dstate <= 128)
        k_gdr_recurrent<T, 16><<<grid, kThreads, 0, st>>>(a);
    else
        k_gdr_recurrent<T, 32><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
