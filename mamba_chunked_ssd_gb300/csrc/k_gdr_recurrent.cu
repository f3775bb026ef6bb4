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
// Four warps walk the tokens; four more stage the next sixteen in shared memory as
// fp32, normalised there where asked, and store the outputs of the last sixteen.
// (With the staging between the tokens of the same four warps a token took 280
// cycles, half of them for it.)  fp32, 2 x 777 tokens of 8 heads of 64 columns, S 64:
// 90 us, 113 ns a token (111 us before the staging had warps of its own).
#include "gated_delta.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 256;  // warps 0-3: recurrence, 4-7: staging
constexpr int kCols = 16;      // columns per block
constexpr int kTok = 16;       // tokens per tile: eight threads stage each token's row

template <int RP>
struct Tile {
    float k[kTok][8 * RP], q[kTok][8 * RP];
    float v[kTok][kCols], y[kTok][kCols];
    float4 c[kTok];  // decay, beta, scale of the output, q . k
};

// RP: state rows per lane (8 lanes span S <= 8 RP rows).
template <typename T, int RP>
__global__ void __launch_bounds__(kThreads) k_gdr_recurrent(const GdrArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Tile<RP>* tiles = reinterpret_cast<Tile<RP>*>(smem);  // [2]
    const Geom& g = a.g;
    const int S = (int)g.dstate, H = (int)g.headdim;
    const int64_t h = blockIdx.y, b = blockIdx.z;
    const int64_t L = g.seqlen, n = row_length(a.lengths, b, L);
    const int64_t grp = h / g.heads_per_group;
    const int col0 = blockIdx.x * kCols;
    const int64_t bh = b * g.nheads + h;
    const int64_t tiles_n = (n + kTok - 1) / kTok;

    if (threadIdx.x < 128) {
        // ------------------------------ recurrence ------------------------------
        const int c = threadIdx.x / 8, rl = threadIdx.x % 8;  // column of the block; rows 32 i + 4 rl + j
        float hs[RP];
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const int s = (i / 4) * 32 + rl * 4 + i % 4;
            hs[i] = (a.init && s < S && col0 + c < H) ? a.init[(bh * S + s) * H + col0 + c] : 0.f;
        }
        __syncthreads();  // the first tile is staged
        for (int64_t it = 0; it < tiles_n; ++it) {
            Tile<RP>& m = tiles[it & 1];
            const int nt = (int)imin64(kTok, n - it * kTok);
            for (int t = 0; t < nt; ++t) {
                const float4 co = m.c[t];
                const float vt = m.v[t][c];
                float kv[RP], r[4] = {0.f, 0.f, 0.f, 0.f}, p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < RP; i += 4) {
                    const float4 k4 = *reinterpret_cast<const float4*>(&m.k[t][(i / 4) * 32 + rl * 4]);
                    kv[i] = k4.x, kv[i + 1] = k4.y, kv[i + 2] = k4.z, kv[i + 3] = k4.w;
                    r[0] = fmaf(k4.x, hs[i], r[0]);
                    r[1] = fmaf(k4.y, hs[i + 1], r[1]);
                    r[2] = fmaf(k4.z, hs[i + 2], r[2]);
                    r[3] = fmaf(k4.w, hs[i + 3], r[3]);
                }
#pragma unroll
                for (int i = 0; i < RP; i += 4) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&m.q[t][(i / 4) * 32 + rl * 4]);
                    p[0] = fmaf(q4.x, hs[i], p[0]);
                    p[1] = fmaf(q4.y, hs[i + 1], p[1]);
                    p[2] = fmaf(q4.z, hs[i + 2], p[2]);
                    p[3] = fmaf(q4.w, hs[i + 3], p[3]);
                }
                float rs = (r[0] + r[1]) + (r[2] + r[3]), ps = (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
                for (int x = 4; x > 0; x >>= 1) {
                    rs += __shfl_xor_sync(0xffffffffu, rs, x);
                    ps += __shfl_xor_sync(0xffffffffu, ps, x);
                }
                const float w = co.y * fmaf(-co.x, rs, vt);
#pragma unroll
                for (int i = 0; i < RP; ++i) hs[i] = fmaf(kv[i], w, co.x * hs[i]);
                if (rl == 0) m.y[t][c] = co.z * fmaf(co.x, ps, co.w * w);
            }
            __syncthreads();
        }
        if (a.final_state && col0 + c < H) {
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                const int s = (i / 4) * 32 + rl * 4 + i % 4;
                if (s < S) a.final_state[(bh * S + s) * H + col0 + c] = hs[i];
            }
        }
        return;
    }

    // -------------------------------- staging --------------------------------
    const int row = (threadIdx.x - 128) / 8, part = threadIdx.x % 8;  // token row, eighth of the row
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
    auto stage = [&](Tile<RP>& m) {
        float kk = 0.f, qq = 0.f, qk = 0.f;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            kk = fmaf(kr[i], kr[i], kk);
            qq = fmaf(qr[i], qr[i], qq);
            qk = fmaf(qr[i], kr[i], qk);
        }
#pragma unroll
        for (int x = 4; x > 0; x >>= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, x);
            qq += __shfl_xor_sync(0xffffffffu, qq, x);
            qk += __shfl_xor_sync(0xffffffffu, qk, x);
        }
        const float nk = a.l2norm ? rsqrtf(kk + a.l2_eps) : 1.f, nq = a.l2norm ? rsqrtf(qq + a.l2_eps) : 1.f;
#pragma unroll
        for (int i = 0; i < RP; i += 4) {
            *reinterpret_cast<float4*>(&m.k[row][(i / 4) * 32 + part * 4]) =
                make_float4(nk * kr[i], nk * kr[i + 1], nk * kr[i + 2], nk * kr[i + 3]);
            *reinterpret_cast<float4*>(&m.q[row][(i / 4) * 32 + part * 4]) =
                make_float4(qr[i], qr[i + 1], qr[i + 2], qr[i + 3]);
        }
        m.v[row][part * 2] = vr[0];
        m.v[row][part * 2 + 1] = vr[1];
        if (part == 0) m.c[row] = make_float4(expf(gr), br, a.scale * nq, qk * nk);
    };
    auto store = [&](const Tile<RP>& m, int64_t t0) {
        if (t0 + row >= n) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int cc = part * 2 + i;
            if (col0 + cc < H) y[(t0 + row) * g.nheads * H + cc] = from_f32<T>(m.y[row][cc]);
        }
    };
    if (tiles_n > 0) {
        fetch(0);
        stage(tiles[0]);
        fetch(kTok);
    }
    __syncthreads();
    for (int64_t it = 0; it < tiles_n; ++it) {
        // beside tile `it`: the outputs before it, then the tile behind it in their place
        if (it > 0) {
            store(tiles[(it + 1) & 1], (it - 1) * kTok);
        }
        if (it + 1 < tiles_n) {
            stage(tiles[(it + 1) & 1]);
            fetch((it + 2) * kTok);
        }
        __syncthreads();
    }
    if (tiles_n > 0) store(tiles[(tiles_n - 1) & 1], (tiles_n - 1) * kTok);
    for (int64_t t = n + row; t < L; t += kTok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int cc = part * 2 + i;
            if (col0 + cc < H) y[t * g.nheads * H + cc] = from_f32<T>(0.f);
        }
    }
}

template <typename T, int RP>
cudaError_t launch_rp(const GdrArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.g.headdim + kCols - 1) / kCols), (unsigned)a.g.nheads, (unsigned)a.g.batch);
    constexpr int smem = 2 * (int)sizeof(Tile<RP>);
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(k_gdr_recurrent<T, RP>), smem);
    if (e != cudaSuccess) return e;
    k_gdr_recurrent<T, RP><<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const GdrArgs& a, cudaStream_t st) {
    if (a.g.dstate <= 64) return launch_rp<T, 8>(a, st);
    if (a.g.dstate <= 128) return launch_rp<T, 16>(a, st);
    return launch_rp<T, 32>(a, st);
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
