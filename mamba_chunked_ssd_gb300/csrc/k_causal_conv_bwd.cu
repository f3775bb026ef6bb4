// k_causal_conv_bwd.cu — gradients of the depthwise causal convolution.  With
// p_t = bias + sum_w weight[w] x_{t - (W - 1) + w}, y_t = act(p_t) and d_t = dy_t act'(p_t):
//
//   dx_t = sum_w weight[w] d_{t + (W - 1) - w}  (+ dfinal of the last W - 1 inputs)
//   dweight[w] = sum_t d_t x_{t - (W - 1) + w},  dbias = sum_t d_t
//
// x and dy are read once and dx is written once.  A thread owns the channels of one vector and
// a run of tokens: it slides a window of W inputs and one of W d's along, so that p is
// computed again from the same loads; d_t is ready W - 1 tokens before dx needs it last, so a
// run reads W - 1 tokens of the next one too.  Inputs come through shared memory, each thread's
// to its own place, 16 tokens ahead.  Sums over a run stay in registers and go to a row of
// partial sums, which a second kernel adds up.  About 22 instructions an element (19 of them packed multiplications
// and additions of two) in 16 warps of an SM bound it next to memory: 4 x 8192 x 8192 in bf16 273 us, 5.9
// TB/s; 4 x 4096 x 8192 in fp32 250 us, 6.4 TB/s.  (Vectors of four bytes, with 24 to 32 warps: 328 and 319 us.)
// Wider than four taps registers leave eight warps: widths 2 to 8 of 4 x 8192 x 8192 in bf16 246, 253, 273, 316, 341, 369,
// 416 us; of 4 x 4096 x 4096 in fp32 128, 131, 132, 133, 143, 146, 159.
#include "glr_math.cuh"

namespace m2 {
namespace {

using glr::add2;
using glr::f2;
using glr::fma2;
using glr::mul2;
using glr::sigmoid2;

constexpr int kThreads = 128;
// Blocks of an SM that registers have to allow.
constexpr int per_sm(int W) { return W <= 4 ? 4 : 2; }
constexpr int kAhead = 8;
// Eights of tokens under way per thread (4 x 8192 x 8192 in bf16: one 293 us, two 273, three 272; 16 x 1024 x 4096 93, 92
// and 93).
constexpr int kDepth = 2;

template <typename T, int VEC>
__device__ __forceinline__ void widen(const typename VecOf<T, VEC>::type& r, float2 (&f)[(VEC + 1) / 2]) {
    float v[VEC];
    unpack<VEC>(r, v, (const T*)nullptr);
#pragma unroll
    for (int i = 0; i < VEC; i += 2) f[i / 2] = make_float2(v[i], i + 1 < VEC ? v[i + 1 < VEC ? i + 1 : i] : 0.f);
}
template <typename T, int VEC>
__device__ __forceinline__ typename VecOf<T, VEC>::type narrow(const float2 (&f)[(VEC + 1) / 2]) {
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
    return pack<T, VEC>(v);
}

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, per_sm(W)) k_causal_conv_bwd(const ConvBwdArgs a, int64_t run) {
    using V = typename VecOf<T, VEC>::type;
    constexpr int N2 = (VEC + 1) / 2;
    tc::griddep_launch_dependents();  // the sum over the runs may be launched; it waits for this grid's end
    const int64_t C = a.channels, c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (c >= C) return;
    const int64_t b = blockIdx.z, t0 = (int64_t)blockIdx.y * run, t1 = imin64(t0 + run, a.seqlen);
    const int64_t n = row_length(a.lengths, b, a.seqlen), m1 = imin64(t1, n);  // tokens t0 .. m1 - 1 are computed
    const T* x = static_cast<const T*>(a.x) + b * a.seqlen * a.x_stride + c;
    const T* dy = static_cast<const T*>(a.dy) + b * a.seqlen * a.dy_stride + c;
    T* dx = static_cast<T*>(a.dx) + b * a.seqlen * a.dx_stride + c;
    const T* init = a.init ? static_cast<const T*>(a.init) + b * (W - 1) * C + c : nullptr;
    const T* dfinal = a.dfinal ? static_cast<const T*>(a.dfinal) + b * (W - 1) * C + c : nullptr;

    float2 wt[W][N2], bias[N2], dw[W][N2], db[N2];
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const bool two = 2 * i + 1 < VEC;
        bias[i] = a.bias ? make_float2(a.bias[c + 2 * i], two ? a.bias[c + 2 * i + 1] : 0.f) : f2(0.f);
        db[i] = f2(0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            wt[w][i] = make_float2(a.weight[(c + 2 * i) * W + w], two ? a.weight[(c + 2 * i + 1) * W + w] : 0.f);
            dw[w][i] = f2(0.f);
        }
    }
    if (t0 < m1 || t0 == 0) {
        float2 xs[W][N2], ds[W][N2];  // xs[w]: the input W - 1 - w tokens back; ds[w]: d w tokens back
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int i = 0; i < N2; ++i) xs[w][i] = ds[w][i] = f2(0.f);
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int64_t t = t0 - (W - 1) + w;
            V v = V{};
            if (t >= 0) v = *reinterpret_cast<const V*>(x + t * a.x_stride);
            else if (init) v = *reinterpret_cast<const V*>(init + (t + W - 1) * C);
            widen<T, VEC>(v, xs[w + 1]);
        }
        // d of the next token, into its window; its products with the window of inputs
        auto token = [&](const V& xv, const V& dv, bool live, bool sum) {
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    xs[w][i] = xs[w + 1][i];
                    ds[W - 1 - w][i] = ds[W - 2 - w][i];
                }
            widen<T, VEC>(xv, xs[W - 1]);
            widen<T, VEC>(dv, ds[0]);
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                if (SILU) {
                    float2 p = bias[i];
#pragma unroll
                    for (int w = 0; w < W; ++w) p = fma2(wt[w][i], xs[w][i], p);
                    const float2 g = sigmoid2(p);  // (act' first: d p could pass the largest number where act' is 1)
                    ds[0][i] = mul2(ds[0][i], mul2(g, fma2(p, fma2(g, f2(-1.f), f2(1.f)), f2(1.f))));
                    if (!live) ds[0][i] = f2(0.f);  // (p of what is not finite)
                }
                if (sum) {
                    db[i] = add2(db[i], ds[0][i]);
#pragma unroll
                    for (int w = 0; w < W; ++w) dw[w][i] = fma2(ds[0][i], xs[w][i], dw[w][i]);
                }
            }
        };
        // the gradient of the input W - 1 tokens back
        auto grad = [&](float2 (&g)[N2]) {
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                g[i] = mul2(wt[0][i], ds[0][i]);
#pragma unroll
                for (int w = 1; w < W; ++w) g[i] = fma2(wt[w][i], ds[w][i], g[i]);
            }
        };
        // the same for a token near a row's end (or before its start), where dfinal adds to it
        auto emit = [&](int64_t u) {
            float2 g[N2];
            grad(g);
            if (dfinal && u >= n - (W - 1)) {
                float2 v[N2];
                widen<T, VEC>(*reinterpret_cast<const V*>(dfinal + (u - n + W - 1) * C), v);
#pragma unroll
                for (int i = 0; i < N2; ++i) g[i] = add2(g[i], v[i]);
            }
            if (u >= 0) *reinterpret_cast<V*>(dx + u * a.dx_stride) = narrow<T, VEC>(g);
            else if (a.dinit)
                *reinterpret_cast<V*>(static_cast<T*>(a.dinit) + (b * (W - 1) + u + W - 1) * C + c) = narrow<T, VEC>(g);
        };
        auto load = [&](const T* p, int64_t stride, int64_t t) { return *reinterpret_cast<const V*>(p + t * stride); };
        const V none = V{};
        // the first W - 1 tokens: what they complete lies before the run (the first one's is the state)
        int64_t s = t0;
#pragma unroll 1
        for (int k = 0; k < W - 1; ++k, ++s) {
            const bool in = s < n, mine = s < m1;
            token(in ? load(x, a.x_stride, s) : none, in ? load(dy, a.dy_stride, s) : none, in, mine);
            if (t0 == 0) emit(s - (W - 1));
        }
        // tokens that complete the gradient of one of this run's, none of them near the row's end
        const int64_t plain = imin64(m1, n - (W - 1)) - s;
        if (plain > 0) {
            const int64_t whole = plain / kAhead;
            if constexpr (sizeof(V) >= 4) {
                __shared__ V ring[2][kDepth * kAhead][kThreads];
                auto ahead = [&](int64_t k) {
                    if (k < whole) {
                        const T *px = x + (s + k * kAhead) * a.x_stride, *pd = dy + (s + k * kAhead) * a.dy_stride;
#pragma unroll
                        for (int u = 0; u < kAhead; ++u) {
                            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(
                                             &ring[0][k % kDepth * kAhead + u][threadIdx.x])),
                                         "l"(px + u * a.x_stride), "n"(sizeof(V))
                                         : "memory");
                            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(
                                             &ring[1][k % kDepth * kAhead + u][threadIdx.x])),
                                         "l"(pd + u * a.dy_stride), "n"(sizeof(V))
                                         : "memory");
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int k = 0; k < kDepth; ++k) ahead(k);
                T* out = dx + (s - (W - 1)) * a.dx_stride;
                for (int64_t k = 0; k < whole; ++k) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        token(ring[0][k % kDepth * kAhead + u][threadIdx.x], ring[1][k % kDepth * kAhead + u][threadIdx.x],
                              true, true);
                        float2 g[N2];
                        grad(g);
                        *reinterpret_cast<V*>(out) = narrow<T, VEC>(g);
                        out += a.dx_stride;
                    }
                    ahead(k + kDepth);
                }
            } else {
                for (int64_t k = 0; k < whole; ++k) {
                    V vx[kAhead], vd[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        vx[u] = load(x, a.x_stride, s + k * kAhead + u);
                        vd[u] = load(dy, a.dy_stride, s + k * kAhead + u);
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        token(vx[u], vd[u], true, true);
                        float2 g[N2];
                        grad(g);
                        *reinterpret_cast<V*>(dx + (s + k * kAhead + u - (W - 1)) * a.dx_stride) = narrow<T, VEC>(g);
                    }
                }
            }
            s += whole * kAhead;
        }
        // the rest of the run, and the W - 1 tokens behind it
#pragma unroll 1
        for (; s < m1 + W - 1; ++s) {
            const bool in = s < n;
            token(in ? load(x, a.x_stride, s) : none, in ? load(dy, a.dy_stride, s) : none, in, s < m1);
            if (s - (W - 1) >= t0 && s - (W - 1) < m1) emit(s - (W - 1));
        }
    }
    for (int64_t t = t0 > n ? t0 : n; t < t1; ++t) *reinterpret_cast<V*>(dx + t * a.dx_stride) = V{};

    float* part = a.partials + ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * C * (W + 1);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int w = 0; w < W; ++w) part[(c + i) * W + w] = i % 2 ? dw[w][i / 2].y : dw[w][i / 2].x;
        part[C * W + c + i] = i % 2 ? db[i / 2].y : db[i / 2].x;
    }
}

// Runs of each row, as blocks that fill the GPU's places whole times, with the least time: that of a run of tokens and
// of about 11 more a tap (the next run's first ones, the weights and the sums), for each filling.  16 x 1024 x 4096 in
// bf16: runs of 256 tokens, of which one filling lacks a sixth, 92 us; of 114, in two whole ones, 95.
int64_t runs_of(int64_t batch, int64_t seqlen, int64_t gx, int width) {
    const int sms = sm_count();
    const int64_t places = per_sm(width) * (int64_t)(sms > 0 ? sms : 152), blocks = gx * batch, most = (seqlen + 31) / 32;
    int64_t best = 1, least = -1;
    for (int64_t waves = 1; waves <= 64; ++waves) {
        int64_t R = waves * places / blocks;
        R = imin64(R < 1 ? 1 : R, most);
        const int64_t time = (R * blocks + places - 1) / places * ((seqlen + R - 1) / R + 11 * width);
        if (least < 0 || time < least) best = R, least = time;
        if (R == most) break;
    }
    return imin64(best, 65535);
}

constexpr int kVecBytes = 8;
template <typename T>
int64_t grid_x(int64_t channels, int vec) {
    return (channels + (int64_t)kThreads * vec - 1) / ((int64_t)kThreads * vec);
}

template <typename T, int VEC, int W>
cudaError_t launch_w(const ConvBwdArgs& a, cudaStream_t st) {
    const int64_t gx = grid_x<T>(a.channels, VEC);
    int64_t R = runs_of(a.batch, a.seqlen, gx, W);
    const int64_t run = (a.seqlen + R - 1) / R;
    R = (a.seqlen + run - 1) / run;
    const dim3 grid((unsigned)gx, (unsigned)R, (unsigned)a.batch);
    if (a.silu) k_causal_conv_bwd<T, VEC, W, true><<<grid, kThreads, 0, st>>>(a, run);
    else k_causal_conv_bwd<T, VEC, W, false><<<grid, kThreads, 0, st>>>(a, run);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_sum_rows(a.partials, R * a.batch, {a.dweight, a.channels * W}, {a.dbias, a.channels}, {}, nullptr, st);
}

template <typename T, int VEC>
cudaError_t launch_v(const ConvBwdArgs& a, cudaStream_t st) {
    switch (a.width) {
        case 2: return launch_w<T, VEC, 2>(a, st);
        case 3: return launch_w<T, VEC, 3>(a, st);
        case 4: return launch_w<T, VEC, 4>(a, st);
        case 5: return launch_w<T, VEC, 5>(a, st);
        case 6: return launch_w<T, VEC, 6>(a, st);
        case 7: return launch_w<T, VEC, 7>(a, st);
        default: return launch_w<T, VEC, 8>(a, st);
    }
}

// The widest vectors on which every row starts, of up to 8 bytes.
template <typename T>
cudaError_t launch_t(const ConvBwdArgs& a, cudaStream_t st) {
    constexpr int VEC = kVecBytes / sizeof(T);
    const uintptr_t p =
        reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dx);
    auto fits = [&](int n) {
        return a.channels % n == 0 && a.x_stride % n == 0 && a.dy_stride % n == 0 && a.dx_stride % n == 0 &&
               p % (n * sizeof(T)) == 0;
    };
    if (fits(VEC)) return launch_v<T, VEC>(a, st);
    if constexpr (VEC == 4)
        if (fits(2)) return launch_v<T, 2>(a, st);
    return launch_v<T, 1>(a, st);
}

}  // namespace

int64_t conv_bwd_partials(int64_t batch, int64_t seqlen, int64_t channels, int width) {
    // whichever vectors the call's alignment allows
    int64_t most = 1;
    for (int vec = 1; vec <= 4; vec *= 2) {
        const int64_t R = runs_of(batch, seqlen, grid_x<float>(channels, vec), width);
        most = R > most ? R : most;
    }
    return most * batch * channels * (width + 1);
}

cudaError_t launch_causal_conv_bwd(const ConvBwdArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
