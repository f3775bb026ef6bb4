// k_gdr_recurrent.cu — the gated delta rule token by token on the CUDA cores,
// for every shape and dtype:
//
//   h <- a h + k (beta (v - a h^T k))^T,  y = scale h^T q,   a = e^g
//
// four tokens at a time.  Columns of the state do not meet, so a block owns 8 to 40
// columns of one head for the whole sequence, and a column's rows lie in the registers
// of eight lanes.  What bounds it is the chain from state to
// state: the sum h^T k over the rows (registers, then three shuffles), the
// correction, the update.  Four tokens share one pass of it: with h the state before
// them, C_ij the decay from token j to token i and A_i the one up to token i,
//   r_i = h^T k_i, p_i = h^T q_i                                 (eight sums at once)
//   w_i = beta_i v_i - beta_i A_i r_i - sum_{j<i} beta_i C_ij (k_i . k_j) w_j
//   y_i = scale (A_i p_i + sum_{j<=i} C_ij (q_i . k_j) w_j)
//   h  <- A_3 h + sum_j C_3j k_j w_j.
// The factors of w_j and r_i do not depend on the state.  Tiles of sixteen tokens go
// through three steps, each a tile behind the other: four warps stage a tile in shared
// memory as fp32, normalised where asked, and form the factors of the one before it,
// while others walk the tokens of the one before that.  fp32, 2 x 777 tokens of 8 heads
// of 64 columns, S 64 (128 blocks): 54 us, 70 ns a token (113 with a pass to a token);
// 4 x 2048 tokens of 32 heads of 128 columns, S 128: 1.43 ms (1.73), bound by the reads of
// k and q from shared memory.
#include "gated_delta.cuh"
#include "tc_ptx.cuh"

namespace m2 {
namespace {

constexpr int kStage = 128;  // threads beside the walkers: eight to a token
constexpr int kTiles = 4;
constexpr int kTok = 16;       // tokens per tile: eight threads stage each token's row

constexpr int kQuad = 4;       // tokens of one pass

template <int RP, int COLS>
struct Tile {
    float k[kTok][8 * RP], q[kTok][8 * RP];
    float v[kTok][COLS], y[kTok][COLS];  // v times beta
    float4 l[kTok];                        // factors of w_0, w_1, w_2 in w, and of r
    float4 s[kTok];                        // factors of w_0 .. w_3 in y
    float f[kTok];                         // factor of p in y
    float4 t[kTok];                        // its decay, beta, scale with q's norm
    float4 d[kTok / kQuad];                // decays from its tokens to the end of the quad
    float a3[kTok / kQuad];                // and of the state before
};

// The sums of eight values over eight neighbouring lanes: value `part` to lane `part`.
__device__ __forceinline__ float sum8(float (&x)[8], int part) {
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) {
        const bool up = (part & m) != 0;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + m], m);
            x[i] = (up ? x[i + m] : x[i]) + other;
        }
    }
    return x[0];
}

// RP: state rows per lane (8 lanes span S <= 8 RP rows).  COLS: columns per block, CPL of them per lane.
template <typename T, int RP, int COLS, int CPL>
__global__ void __launch_bounds__(8 * COLS / CPL + kStage) k_gdr_recurrent(const GdrArgs a) {
    constexpr bool kKeep = RP * CPL <= 16;  // k stays in registers from the sums to the update
    extern __shared__ __align__(16) uint8_t smem[];
    Tile<RP, COLS>* tiles = reinterpret_cast<Tile<RP, COLS>*>(smem);  // [kTiles]
    const Geom& g = a.g;
    const int S = (int)g.dstate, H = (int)g.headdim;
    const int64_t h = blockIdx.y, b = blockIdx.z;
    const int64_t L = g.seqlen, n = row_length(a.lengths, b, L);
    const int64_t grp = h / g.heads_per_group;
    const int col0 = blockIdx.x * COLS;
    const int64_t bh = b * g.nheads + h;
    const int64_t tiles_n = (n + kTok - 1) / kTok;

    if (threadIdx.x < 8 * COLS / CPL) {
        // ------------------------------ recurrence ------------------------------
        const int c = threadIdx.x / 8 * CPL, rl = threadIdx.x % 8;  // first column in the block; rows 32 i + 4 rl + j
        float2 hs[CPL][RP / 2];
#pragma unroll
        for (int e = 0; e < CPL; ++e)
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                const int s = (i / 4) * 32 + rl * 4 + i % 4;
                const float x = (a.init && s < S && col0 + c + e < H) ? a.init[(bh * S + s) * H + col0 + c + e] : 0.f;
                if (i & 1) hs[e][i / 2].y = x;
                else hs[e][i / 2].x = x;
            }
        __syncthreads();  // the first tile is staged
        __syncthreads();  // and has its factors
        // the quad's k and q (kKeep)
        constexpr int kHeld = kKeep ? RP / 2 : 1;
        float2 kv[kQuad][kHeld], qv[kQuad][kHeld];
        auto load = [&](float2(&to)[kQuad][kHeld], const float(*from)[8 * RP]) {
#pragma unroll
            for (int x = 0; x < kQuad; ++x)
#pragma unroll
                for (int i = 0; i < (kKeep ? RP : 0); i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&from[x][(i / 4) * 32 + rl * 4]);
                    to[x][i / 2] = make_float2(f.x, f.y);
                    to[x][i / 2 + 1] = make_float2(f.z, f.w);
                }
        };
        // rows i .. i + 3 of this lane of token x
        auto rows4 = [&](const float2(&held)[kQuad][kHeld], const float(*from)[8 * RP], int x, int i, float2& f0, float2& f1) {
            if (kKeep) {
                f0 = held[x][kKeep ? i / 2 : 0];
                f1 = held[x][kKeep ? i / 2 + 1 : 0];
            } else {
                const float4 f = *reinterpret_cast<const float4*>(&from[x][(i / 4) * 32 + rl * 4]);
                f0 = make_float2(f.x, f.y);
                f1 = make_float2(f.z, f.w);
            }
        };
        load(kv, tiles[0].k);
        load(qv, tiles[0].q);
        for (int64_t it = 0; it < tiles_n; ++it) {
            Tile<RP, COLS>& m = tiles[it % kTiles];
            const Tile<RP, COLS>& next = tiles[(it + 1) % kTiles];
            const int nt = (int)imin64(kTok, n - it * kTok);
#pragma unroll 1
            for (int t = 0; t < nt; t += kQuad) {  // (tokens past the end are staged as zeros, without decay)
                float r[CPL][kQuad], p[CPL][kQuad], w[CPL][kQuad];
                auto sums = [&](const float2(&held)[kQuad][kHeld], const float(*from)[8 * RP], float(&o)[CPL][kQuad]) {
                    float2 acc[CPL][kQuad];
#pragma unroll
                    for (int x = 0; x < kQuad; ++x)
#pragma unroll
                        for (int e = 0; e < CPL; ++e) acc[e][x] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < RP; i += 4)
#pragma unroll
                        for (int x = 0; x < kQuad; ++x) {
                            float2 f0, f1;
                            rows4(held, from, x, i, f0, f1);
#pragma unroll
                            for (int e = 0; e < CPL; ++e) {
                                acc[e][x] = tc::fma_f32x2(f0, hs[e][i / 2], acc[e][x]);
                                acc[e][x] = tc::fma_f32x2(f1, hs[e][i / 2 + 1], acc[e][x]);
                            }
                        }
#pragma unroll
                    for (int x = 0; x < kQuad; ++x)
#pragma unroll
                        for (int e = 0; e < CPL; ++e) o[e][x] = acc[e][x].x + acc[e][x].y;
                };
                sums(kv, m.k + t, r);
#pragma unroll
                for (int m8 = 4; m8 > 0; m8 >>= 1)
#pragma unroll
                    for (int x = 0; x < kQuad; ++x)
#pragma unroll
                        for (int e = 0; e < CPL; ++e) r[e][x] += __shfl_xor_sync(0xffffffffu, r[e][x], m8);
                sums(qv, m.q + t, p);
#pragma unroll
                for (int x = 0; x < kQuad; ++x) {
                    const float4 l = m.l[t + x];
#pragma unroll
                    for (int e = 0; e < CPL; ++e) {
                        w[e][x] = fmaf(l.w, r[e][x], m.v[t + x][c + e]);
                        if (x > 0) w[e][x] = fmaf(l.x, w[e][0], w[e][x]);
                        if (x > 1) w[e][x] = fmaf(l.y, w[e][1], w[e][x]);
                        if (x > 2) w[e][x] = fmaf(l.z, w[e][2], w[e][x]);
                    }
                }
                const float4 d = m.d[t / kQuad];
                const float a3 = m.a3[t / kQuad];
#pragma unroll
                for (int e = 0; e < CPL; ++e)
#pragma unroll
                    for (int i = 0; i < RP / 2; ++i) hs[e][i] = tc::mul_f32x2(make_float2(a3, a3), hs[e][i]);
#pragma unroll
                for (int x = 0; x < kQuad; ++x) {
                    const float dx = x == 0 ? d.x : x == 1 ? d.y : x == 2 ? d.z : d.w;
#pragma unroll
                    for (int i = 0; i < RP; i += 4) {
                        float2 f0, f1;
                        rows4(kv, m.k + t, x, i, f0, f1);
#pragma unroll
                        for (int e = 0; e < CPL; ++e) {
                            const float2 u = make_float2(w[e][x] * dx, w[e][x] * dx);
                            hs[e][i / 2] = tc::fma_f32x2(f0, u, hs[e][i / 2]);
                            hs[e][i / 2 + 1] = tc::fma_f32x2(f1, u, hs[e][i / 2 + 1]);
                        }
                    }
                }
                // the next quad's k and q, while the outputs of this one are summed (behind the last tile, whatever
                // is there: the loads stay inside the tiles)
                const bool last = t + kQuad >= kTok;
                load(kv, last ? next.k : m.k + t + kQuad);
                load(qv, last ? next.q : m.q + t + kQuad);
                // p of one token (and one column) to each lane or two; y takes no w of a later token, whatever it is
                float ps, ws[kQuad];
                int mine, col = c;
                if constexpr (CPL == 2) {
                    mine = rl & 3;
                    col += rl >> 2;
                    float both[8];
#pragma unroll
                    for (int x = 0; x < kQuad; ++x) {
                        both[x] = p[0][x], both[4 + x] = p[1][x];
                        ws[x] = rl & 4 ? w[1][x] : w[0][x];
                    }
                    ps = sum8(both, rl);
                } else {
                    mine = rl >> 1;
#pragma unroll
                    for (int x = 0; x < kQuad; ++x) ws[x] = w[0][x];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float other = __shfl_xor_sync(0xffffffffu, mine & 2 ? p[0][x] : p[0][x + 2], 4);
                        p[0][x] = (mine & 2 ? p[0][x + 2] : p[0][x]) + other;
                    }
                    const float other = __shfl_xor_sync(0xffffffffu, mine & 1 ? p[0][0] : p[0][1], 2);
                    ps = (mine & 1 ? p[0][1] : p[0][0]) + other;
                    ps += __shfl_xor_sync(0xffffffffu, ps, 1);
                }
                const float4 sm = m.s[t + mine];
                float out = fmaf(sm.x, ws[0], m.f[t + mine] * ps);
                out = fmaf(sm.y, mine > 0 ? ws[1] : 0.f, out);
                out = fmaf(sm.z, mine > 1 ? ws[2] : 0.f, out);
                out = fmaf(sm.w, mine > 2 ? ws[3] : 0.f, out);
                if (CPL == 2 || (rl & 1) == 0) m.y[t + mine][col] = out;
            }
            __syncthreads();
        }
        if (a.final_state) {
#pragma unroll
            for (int e = 0; e < CPL; ++e)
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    const int s = (i / 4) * 32 + rl * 4 + i % 4;
                    if (s < S && col0 + c + e < H)
                        a.final_state[(bh * S + s) * H + col0 + c + e] = i & 1 ? hs[e][i / 2].y : hs[e][i / 2].x;
                }
        }
        return;
    }

    // ---------------------- staging, factors and outputs ----------------------
    const int row = (threadIdx.x - 8 * COLS / CPL) / 8, part = threadIdx.x % 8;  // token row, eighth of the row
    const T* q = static_cast<const T*>(a.q) + b * L * a.q_stride + grp * S;
    const T* k = static_cast<const T*>(a.k) + b * L * a.k_stride + grp * S;
    const T* v = static_cast<const T*>(a.v) + b * L * a.v_stride + h * H + col0;
    T* y = static_cast<T*>(a.y) + (b * L * g.nheads + h) * H + col0;
    float kr[RP], qr[RP], vr[COLS / 8], gr, br;
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
        for (int i = 0; i < COLS / 8; ++i) {
            const int cc = part * (COLS / 8) + i;
            vr[i] = (t < n && col0 + cc < H) ? to_f32(v[t * a.v_stride + cc]) : 0.f;
        }
        gr = t < n ? a.gate[(b * L + t) * g.nheads + h] : 0.f;
        br = t < n ? a.beta[(b * L + t) * g.nheads + h] : 0.f;
    };
    auto stage = [&](Tile<RP, COLS>& m) {
        float nk = 1.f, nq = 1.f;
        if (a.l2norm) {
            float kk = 0.f, qq = 0.f;
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                kk = fmaf(kr[i], kr[i], kk);
                qq = fmaf(qr[i], qr[i], qq);
            }
#pragma unroll
            for (int x = 4; x > 0; x >>= 1) {
                kk += __shfl_xor_sync(0xffffffffu, kk, x);
                qq += __shfl_xor_sync(0xffffffffu, qq, x);
            }
            nk = rsqrtf(kk + a.l2_eps);
            nq = rsqrtf(qq + a.l2_eps);
        }
#pragma unroll
        for (int i = 0; i < RP; i += 4) {
            *reinterpret_cast<float4*>(&m.k[row][(i / 4) * 32 + part * 4]) =
                make_float4(nk * kr[i], nk * kr[i + 1], nk * kr[i + 2], nk * kr[i + 3]);
            *reinterpret_cast<float4*>(&m.q[row][(i / 4) * 32 + part * 4]) =
                make_float4(qr[i], qr[i + 1], qr[i + 2], qr[i + 3]);
        }
#pragma unroll
        for (int i = 0; i < COLS / 8; ++i) m.v[row][part * (COLS / 8) + i] = br * vr[i];
        if (part == 0) m.t[row] = make_float4(expf(gr), br, a.scale * nq, 0.f);
    };
    auto factors = [&](Tile<RP, COLS>& m) {
        // a warp's four rows are a quad: token `mine` of it meets k of all four (those not before it are left out below)
        const int mine = row & 3, quad = row >> 2;
        float2 kk[kQuad], qk[kQuad];
#pragma unroll
        for (int j = 0; j < kQuad; ++j) kk[j] = qk[j] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RP; i += 4) {
            const int at = (i / 4) * 32 + part * 4;
            const float4 k4 = *reinterpret_cast<const float4*>(&m.k[row][at]);
            const float4 q4 = *reinterpret_cast<const float4*>(&m.q[row][at]);
#pragma unroll
            for (int j = 0; j < kQuad; ++j) {
                const float4 o = *reinterpret_cast<const float4*>(&m.k[4 * quad + j][at]);
                kk[j] = tc::fma_f32x2(make_float2(k4.x, k4.y), make_float2(o.x, o.y), kk[j]);
                kk[j] = tc::fma_f32x2(make_float2(k4.z, k4.w), make_float2(o.z, o.w), kk[j]);
                qk[j] = tc::fma_f32x2(make_float2(q4.x, q4.y), make_float2(o.x, o.y), qk[j]);
                qk[j] = tc::fma_f32x2(make_float2(q4.z, q4.w), make_float2(o.z, o.w), qk[j]);
            }
        }
        float x[8];
#pragma unroll
        for (int j = 0; j < kQuad; ++j) x[j] = kk[j].x + kk[j].y, x[4 + j] = qk[j].x + qk[j].y;
        const float dot = sum8(x, part);  // k . k_j on the first four lanes, q . k_j on the others, j = part % 4
        const int j = part & 3;
        const float4 own = m.t[row];
        float to = 1.f, all = 1.f, end = 1.f;  // decays from token j to this one, up to this one, from this one on
#pragma unroll
        for (int i = 0; i < kQuad; ++i) {
            const float ai = m.t[4 * quad + i].x;
            if (i <= mine) all *= ai;
            if (i <= mine && i > j) to *= ai;
            if (i > mine) end *= ai;
        }
        if (part < 3) reinterpret_cast<float*>(&m.l[row])[part] = j < mine ? -own.y * to * dot : 0.f;
        if (part == 3) {
            m.l[row].w = -own.y * all;
            m.f[row] = own.z * all;
            reinterpret_cast<float*>(&m.d[quad])[mine] = end;
            if (mine == 3) m.a3[quad] = all;
        }
        if (part > 3) reinterpret_cast<float*>(&m.s[row])[j] = j <= mine ? own.z * to * dot : 0.f;
    };
    auto store = [&](const Tile<RP, COLS>& m, int64_t t0) {
        if (t0 + row >= n) return;
#pragma unroll
        for (int i = 0; i < COLS / 8; ++i) {
            const int cc = part * (COLS / 8) + i;
            if (col0 + cc < H) y[(t0 + row) * g.nheads * H + cc] = from_f32<T>(m.y[row][cc]);
        }
    };
    fetch(0);
    for (int64_t it = -2; it < tiles_n; ++it) {
        // beside the walk of tile `it`: the factors of the next, the outputs of the last, and the tile after next
        if (it >= -1) {
            if (it + 1 < tiles_n) factors(tiles[(it + 1) % kTiles]);
            if (it > 0) store(tiles[(it - 1) % kTiles], (it - 1) * kTok);
        }
        if (it + 2 < tiles_n) {
            stage(tiles[(it + 2) % kTiles]);
            fetch((it + 3) * kTok);
        }
        __syncthreads();
    }
    if (tiles_n > 0) store(tiles[(tiles_n - 1) % kTiles], (tiles_n - 1) * kTok);
    for (int64_t t = n + row; t < L; t += kTok) {
#pragma unroll
        for (int i = 0; i < COLS / 8; ++i) {
            const int cc = part * (COLS / 8) + i;
            if (col0 + cc < H) y[t * g.nheads * H + cc] = from_f32<T>(0.f);
        }
    }
}

template <typename T, int RP, int COLS, int CPL>
cudaError_t launch_k(const GdrArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.g.headdim + COLS - 1) / COLS), (unsigned)a.g.nheads, (unsigned)a.g.batch);
    constexpr int smem = kTiles * (int)sizeof(Tile<RP, COLS>);
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(k_gdr_recurrent<T, RP, COLS, CPL>), smem);
    if (e != cudaSuccess) return e;
    k_gdr_recurrent<T, RP, COLS, CPL><<<grid, 8 * COLS / CPL + kStage, smem, st>>>(a);
    return cudaGetLastError();
}

// As few columns to a block as leave one block to an SM; from there on the shared
// memory's reads count, and two columns to a lane halve them.  1024 tokens in fp32, H 64,
// us with 8 columns / 16 / 32 (two to a lane) to a block: S 64, 16 heads 93 / 105 / 135, 32
// heads 123 / 107 / 135, 64 heads 272 / 178 / 135; S 256 207 / 268 / 327, 397 / 265 / 326,
// 773 / 512 / 325.  40 columns where they leave fewer over than 32 (19 x 637 tokens of 24 heads
// of 40 columns, S 128, fp32: 485 us, with 32 689).
template <typename T, int RP>
cudaError_t launch_rp(const GdrArgs& a, cudaStream_t st) {
    const int sms = sm_count();
    const int64_t fit = sms > 0 ? sms : 152, heads = a.g.batch * a.g.nheads;
    if (heads * ((a.g.headdim + 7) / 8) <= fit) return launch_k<T, RP, 8, 1>(a, st);
    if (heads * ((a.g.headdim + 15) / 16) <= fit) return launch_k<T, RP, 16, 1>(a, st);
    const auto blocks = [&](int n) { return (a.g.headdim + n - 1) / n * n; };
    return blocks(40) < blocks(32) ? launch_k<T, RP, 40, 2>(a, st) : launch_k<T, RP, 32, 2>(a, st);
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
