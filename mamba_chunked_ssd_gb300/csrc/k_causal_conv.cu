// k_causal_conv.cu — depthwise causal convolution over time, channels last,
// with an optional SiLU: over whole sequences, and one token at a time.
//
//   y_t = act(bias + sum_{w < W} weight[c, w] x_{t - (W - 1) + w})
//
// Each input is read once and each output written once: the kernels are bound
// by memory.  A thread owns the channels of one vector and a run of consecutive
// tokens, and slides a window of the last W - 1 inputs through its registers, so a
// token's input is loaded once per run (plus the W - 1 tokens before the run,
// which the neighbouring run has just brought into L2).  Inputs come through
// shared memory, each thread's to its own place, two or three times eight tokens ahead.
// 4 x 8192 tokens of 8192 channels in bf16, width 4, SiLU: 165 us, 6.5 TB/s (0.97 of a plain
// copy; 366 us without loads ahead, 180 with eight in registers; 162 where the variants
// below were compared).  One token of 256
// sequences of these channels: 5.0 us in a graph, from L2 (alone the host's call is the
// time).
#include "gated_delta.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 128;  // tokens per thread, less where that leaves too few blocks
// Tokens whose loads are issued together: 32 where a thread's are of 2 bytes and come through
// registers (14 x 3053 tokens of 823 channels in bf16: 39 us, 16 49, 8 62).
template <typename V>
constexpr int kAheadOf = sizeof(V) < 4 ? 32 : 8;
// Groups of these under way per thread (4 x 8192 x 8192 in bf16: 3 162 us, 2 163, one in
// registers 180; 16 x 1024 x 4096 46 / 50 / 55; 4 x 4096 x 8192 in fp32 177 / 170 / 172).
template <typename T>
constexpr int kDepthOf = sizeof(T) == 2 ? 3 : 2;

// The weights of VEC neighbouring channels: one run of VEC W floats, in 16-byte
// loads where that is whole ones.
template <int VEC, int W>
__device__ __forceinline__ void load_weights(const float* weight, int64_t c, float (&wt)[W][VEC]) {
    float f[VEC * W];
    if (VEC * W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC * W; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(weight + c * W + i);
            f[i] = v.x;
            if (i + 1 < VEC * W) f[i + 1] = v.y;
            if (i + 2 < VEC * W) f[i + 2] = v.z;
            if (i + 3 < VEC * W) f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC * W; ++i) f[i] = weight[c * W + i];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int w = 0; w < W; ++w) wt[w][i] = f[i * W + w];
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads, VEC * W <= 16 ? 5 : 1) k_causal_conv(const ConvArgs a, int run) {
    using V = typename VecOf<T, VEC>::type;
    constexpr int kAhead = kAheadOf<V>;
    const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (c >= a.channels) return;
    const int64_t b = blockIdx.z;
    const int64_t n = row_length(a.lengths, b, a.seqlen);
    const T* x = static_cast<const T*>(a.x) + b * a.seqlen * a.x_stride + c;
    T* y = static_cast<T*>(a.y) + b * a.seqlen * a.y_stride + c;
    const T* init = a.init ? static_cast<const T*>(a.init) + b * (W - 1) * a.channels + c : nullptr;

    // the input at token t < n, from the initial state where t < 0
    auto input = [&](int64_t t) -> V {
        if (t >= 0) return *reinterpret_cast<const V*>(x + t * a.x_stride);
        if (init) return *reinterpret_cast<const V*>(init + (t + W - 1) * a.channels);
        return V{};
    };

    if (blockIdx.y == 0 && a.final_state) {
        T* fin = static_cast<T*>(a.final_state) + b * (W - 1) * a.channels + c;
#pragma unroll
        for (int w = 0; w < W - 1; ++w) *reinterpret_cast<V*>(fin + w * a.channels) = input(n - (W - 1) + w);
    }

    float wt[W][VEC], bias[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.f;
    load_weights<VEC, W>(a.weight, c, wt);

    for (int64_t t0 = (int64_t)blockIdx.y * run; t0 < a.seqlen; t0 += (int64_t)gridDim.y * run) {
        const int64_t t1 = imin64(t0 + run, a.seqlen);
        const int m = (int)(imin64(t1, n) - t0);  // tokens that are computed (none: m <= 0)
        if (m > 0) {
            float win[W][VEC];  // win[w]: the input W - 1 - w tokens back
#pragma unroll
            for (int w = 0; w < W - 1; ++w) unpack<VEC>(input(t0 - (W - 1) + w), win[w + 1], (const T*)nullptr);
            const T* xt = x + t0 * a.x_stride;
            T* yt = y + t0 * a.y_stride;
            auto token = [&](const V& in) {
#pragma unroll
                for (int w = 0; w < W - 1; ++w)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) win[w][i] = win[w + 1][i];
                unpack<VEC>(in, win[W - 1], (const T*)nullptr);
                float s[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    s[i] = bias[i];
#pragma unroll
                    for (int w = 0; w < W; ++w) s[i] = fmaf(wt[w][i], win[w][i], s[i]);
                    if (a.silu) s[i] = silu_f32<T>(s[i]);
                }
                *reinterpret_cast<V*>(yt) = pack<T, VEC>(s);
                yt += a.y_stride;
            };
            const int whole = m / kAhead;
            if constexpr (sizeof(V) >= 4) {
                constexpr int kDepth = kDepthOf<T>;
                // the loads of the next kDepth times eight tokens are under way, each thread's to its own place
                __shared__ V ring[kDepth * kAhead][kThreads];
                auto ahead = [&](int k) {
                    if (k < whole) {
                        const T* from = x + (t0 + (int64_t)k * kAhead) * a.x_stride;
#pragma unroll
                        for (int u = 0; u < kAhead; ++u)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                                             (uint32_t)__cvta_generic_to_shared(&ring[k % kDepth * kAhead + u][threadIdx.x])),
                                         "l"(from + u * a.x_stride), "n"(sizeof(V))
                                         : "memory");
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int k = 0; k < kDepth; ++k) ahead(k);
                for (int k = 0; k < whole; ++k) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
                    V in[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) in[u] = ring[k % kDepth * kAhead + u][threadIdx.x];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) token(in[u]);
                    ahead(k + kDepth);
                }
                xt += (int64_t)whole * kAhead * a.x_stride;
            } else {
                V next[kAhead];
                if (whole > 0) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) next[u] = *reinterpret_cast<const V*>(xt + u * a.x_stride);
                }
                for (int k = 0; k < whole; ++k) {
                    V in[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) in[u] = next[u];
                    xt += kAhead * a.x_stride;
                    if (k + 1 < whole) {
#pragma unroll
                        for (int u = 0; u < kAhead; ++u) next[u] = *reinterpret_cast<const V*>(xt + u * a.x_stride);
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) token(in[u]);
                }
            }
            int left = m - whole * kAhead;
            if (kAhead > 8) {
#pragma unroll 1
                for (; left >= 8; left -= 8) {
                    V in[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) in[u] = *reinterpret_cast<const V*>(xt + u * a.x_stride);
                    xt += 8 * a.x_stride;
#pragma unroll
                    for (int u = 0; u < 8; ++u) token(in[u]);
                }
            }
#pragma unroll 1
            for (; left > 0; --left, xt += a.x_stride) token(*reinterpret_cast<const V*>(xt));
        }
        for (int64_t t = t0 + (m > 0 ? m : 0); t < t1; ++t) *reinterpret_cast<V*>(y + t * a.y_stride) = V{};
    }
}

// One token: a thread reads its channels' state and input, and writes the
// output and the state moved on by one (in place is safe: it reads all of its
// own elements first).  It takes `rows` batch rows, for which it loads its weights
// once: they are as many bytes as a row's data.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) k_causal_conv_step(const ConvArgs a, int rows) {
    using V = typename VecOf<T, VEC>::type;
    const int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (c >= a.channels) return;
    float wt[W][VEC], bias[VEC];
    load_weights<VEC, W>(a.weight, c, wt);
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.f;
    const int64_t b0 = (int64_t)blockIdx.y * rows, b1 = imin64(b0 + rows, a.batch);
#pragma unroll 2
    for (int64_t b = b0; b < b1; ++b) {
        const int64_t at = b * (W - 1) * a.channels + c;
        V in[W];
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
            in[w] = a.init ? *reinterpret_cast<const V*>(static_cast<const T*>(a.init) + at + w * a.channels) : V{};
        in[W - 1] = *reinterpret_cast<const V*>(static_cast<const T*>(a.x) + b * a.x_stride + c);
        float s[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = bias[i];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float f[VEC];
            unpack<VEC>(in[w], f, (const T*)nullptr);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[i] = fmaf(wt[w][i], f[i], s[i]);
        }
#pragma unroll
        for (int w = 0; w < W - 1; ++w)
            *reinterpret_cast<V*>(static_cast<T*>(a.final_state) + at + w * a.channels) = in[w + 1];
        if (a.silu) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[i] = silu_f32<T>(s[i]);
        }
        *reinterpret_cast<V*>(static_cast<T*>(a.y) + b * a.y_stride + c) = pack<T, VEC>(s);
    }
}

template <typename T, int VEC, int W>
cudaError_t launch_w(const ConvArgs& a, bool step, cudaStream_t st) {
    const unsigned gx = (unsigned)((a.channels + (int64_t)kThreads * VEC - 1) / (kThreads * VEC));
    if constexpr (VEC <= 2) {
        if (step) {
            // rows per thread: as many as leave eight blocks to an SM, at most 16
            const int sms = sm_count();
            const int64_t fill = a.batch * gx / (8 * (int64_t)(sms > 0 ? sms : 152));
            const int rows = (int)(fill < 1 ? 1 : imin64(fill, 16));
            k_causal_conv_step<T, VEC, W>
                <<<dim3(gx, (unsigned)((a.batch + rows - 1) / rows)), kThreads, 0, st>>>(a, rows);
        }
    }
    if (!step) {
        constexpr int least = VEC * sizeof(T) < 4 ? 32 : 16;
        // Runs of 128 tokens (4 x 8192 x 8192: 162 us, 64: 162, 256: 166; width 8 110, 124, 105), halved down to
        // 16 (or the 32 that are loaded together) while there are fewer than four blocks to an SM.
        const int sms = sm_count();
        int run = kRun;
        while (run > least && gx * a.batch * ((a.seqlen + run - 1) / run) < 4 * (int64_t)(sms > 0 ? sms : 152)) run /= 2;
        const int64_t runs = (a.seqlen + run - 1) / run;
        k_causal_conv<T, VEC, W>
            <<<dim3(gx, (unsigned)imin64(runs, 65535), (unsigned)a.batch), kThreads, 0, st>>>(a, run);
    }
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_v(const ConvArgs& a, bool step, cudaStream_t st) {
    switch (a.width) {
        case 2: return launch_w<T, VEC, 2>(a, step, st);
        case 3: return launch_w<T, VEC, 3>(a, step, st);
        case 4: return launch_w<T, VEC, 4>(a, step, st);
        case 5: return launch_w<T, VEC, 5>(a, step, st);
        case 6: return launch_w<T, VEC, 6>(a, step, st);
        case 7: return launch_w<T, VEC, 7>(a, step, st);
        default: return launch_w<T, VEC, 8>(a, step, st);
    }
}

// The widest vectors on which every row of x and y starts, of up to 8 bytes over whole
// sequences (registers for eight channels of weights, window and loads under way would
// leave too few warps; 14 x 3053 tokens in bf16: 820 channels 33 us, 822 in pairs 37, 823 one by one 39),
// and pairs for one token, whose weights then come in whole lines and not once for every
// row (256 x 8192 in bf16: pairs 5.0 us, fours 5.4, eights 11.4, one by one 6.2; in fp32 7.2,
// fours 7.7, one by one 7.4).
template <typename T>
cudaError_t launch_t(const ConvArgs& a, bool step, cudaStream_t st) {
    constexpr int VEC = 8 / sizeof(T);
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
    auto fits = [&](int n) {
        return a.channels % n == 0 && a.x_stride % n == 0 && a.y_stride % n == 0 && p % (n * sizeof(T)) == 0;
    };
    if (!step && fits(VEC)) return launch_v<T, VEC>(a, step, st);
    return fits(2) ? launch_v<T, 2>(a, step, st) : launch_v<T, 1>(a, step, st);
}

}  // namespace

cudaError_t launch_causal_conv(const ConvArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, false, st) : launch_t<float>(a, false, st);
}
cudaError_t launch_causal_conv_step(const ConvArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, true, st) : launch_t<float>(a, true, st);
}

}  // namespace m2
