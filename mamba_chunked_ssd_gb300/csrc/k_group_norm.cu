// k_group_norm.cu — group norm over each row's groups of channels, with a gate
// or an activation:
//
//   u = x [SiLU(z)];  u -= mean(u) [if asked];  y = w u / sqrt(mean(u^2) + eps) + bias;
//   y *= SiLU(z), or y = SiLU(y) [if asked]
//
// x (and z) are read once and y is written once: the kernel is bound by
// memory.  A group lives in the registers of TPG threads (a part of a warp, a
// warp, or a block), so the mean and then the squares of the differences from
// it are summed from registers, in fp32 and a fixed order, without a second
// read.  Threads keep their channels and walk down the rows: up to 16 channels to
// a thread, the weights stay in registers and a row's loads are under way while
// the row before is summed.  32768 x 4096 in bf16, groups of 64, gated: 129 us, 6.2 TB/s
// (0.93 of a plain copy; 217 us with a block to a row); 8192 x 4096 in one group,
// gated first: 37 us, 5.4 TB/s (0.81; a block-wide sum a row).
#include "gated_delta.cuh"
#include "mamba2_gated_delta.h"

namespace m2 {
namespace {

constexpr int kWarpBlock = 256;  // threads of a block whose groups stay inside warps

// Sum over the group's threads.  Block-wide, the partial sums go through one of two places in
// turn, so that one barrier is enough: whoever writes a place has met, since it was read,
// at the barrier of the sum between.
template <int TPG>
__device__ __forceinline__ float group_sum(float v, float (*smem)[32], int& turn) {
#pragma unroll
    for (int m = (TPG < 32 ? TPG : 32) / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if constexpr (TPG > 32) {
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) smem[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        v = smem[turn][threadIdx.x & 31 & (TPG / 32 - 1)];
#pragma unroll
        for (int m = TPG / 64; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    }
    return v;
}

// Blocks of an SM that the registers have to allow: 1024 threads for up to eight channels
// to a thread (32768 x 4096 in groups of 64, gated: 130 us, 768 threads 144; 8192 x 2052 in
// fp32 in one group, gated: 41 us, 512 threads 55) and in blocks of 512 (4096 x 8192 in bf16,
// gated: 36 us, 512 threads 38), else 768 for 16 channels (8192 x 4096 in one group, gated,
// without the ring below: 39 us, 1024 threads 49, 512 40).
constexpr int min_blocks(int channels, int tpg) {
    return tpg > 512 || channels > 16 ? 1 : (channels <= 8 || tpg == 512 ? 1024 : 768) / (tpg > 32 ? tpg : kWarpBlock);
}

// bf16 rows come through a ring in shared memory, two or three rows ahead, each thread copying
// what it reads itself: registers hold too few loads for the sums between them.  us without /
// with: blocks, gated before, 2048 channels 36.6 / 33.8, 4096 36.7 / 34.9, 16384 50 / 41 (over
// 28 sizes and modes 6 % faster; two rows ahead are 4 % slower); groups inside warps, 32768 x
// 4096 in groups of 64, gated after 129 / 125 (where they were compared in turn; 129 with
// the ring in later runs), no gate 99 / 85 (three rows 131, 86), but in 8-byte vectors
// 242 / 272.  In fp32 it is slower (1024 channels, gated after, 31 / 37).
constexpr int ring_rows(int tpg) { return tpg > 32 ? 3 : 2; }
template <typename T>
constexpr bool use_ring(int vec, int nv, int tpg) {
    return sizeof(T) == 2 && vec >= (tpg > 32 ? 4 : 8) && nv * vec <= 16 && nv * tpg <= 2048;
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool live) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0) : "memory");
}

// VEC elements per load, NV loads per thread, TPG threads per group.  Groups
// inside warps: a block spans 2^across groups of a row and as many rows as are
// left of its threads.
template <typename T, int VEC, int NV, int TPG>
__global__ void __launch_bounds__(TPG > 32 ? TPG : kWarpBlock, min_blocks(NV * VEC, TPG))
k_group_norm(const NormArgs a, int across) {
    using V = typename VecOf<T, VEC>::type;
    __shared__ float smem[2][32];
    int turn = 0;
    constexpr bool kKeep = NV * VEC <= 16;
    const int lane = threadIdx.x % TPG, slot = threadIdx.x / TPG;
    const int rows_per = TPG > 32 ? 1 : (kWarpBlock / TPG) >> across;
    const int64_t grp = ((int64_t)blockIdx.x << across) + (slot & ((1 << across) - 1));
    const bool mine = grp < a.ngroups;  // the others stay for the warp's shuffles
    const int size = (int)(a.channels / a.ngroups), nvec = size / VEC;
    const int64_t c0 = (mine ? grp : 0) * size;
    const bool before = (a.flags & MAMBA2_NORM_GATE_BEFORE) != 0, after = (a.flags & MAMBA2_NORM_GATE_AFTER) != 0;
    const bool gated = before || after;
    const T* x = static_cast<const T*>(a.x) + c0;
    const T* z = static_cast<const T*>(a.z) + c0;
    T* y = static_cast<T*>(a.y) + c0;

    float w[kKeep ? NV : 1][VEC];
    auto weights = [&](int j, float (&f)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = a.weight && j < nvec ? a.weight[c0 + (int64_t)j * VEC + e] : 1.f;
    };
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < NV; ++i) weights(lane + i * TPG, w[kKeep ? i : 0]);
    }

    int64_t row = (int64_t)blockIdx.y * rows_per + (slot >> across);
    const int64_t step = (int64_t)gridDim.y * rows_per;
    V xr[NV], zr[NV];
    auto load = [&](int64_t r) {
        const bool live = mine && r < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * TPG;
            xr[i] = V{};
            if (live && j < nvec) xr[i] = *reinterpret_cast<const V*>(x + r * a.x_stride + (int64_t)j * VEC);
        }
        if (gated) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = lane + i * TPG;
                zr[i] = V{};
                if (live && j < nvec) zr[i] = *reinterpret_cast<const V*>(z + r * a.z_stride + (int64_t)j * VEC);
            }
        }
    };
    constexpr bool kUseRing = use_ring<T>(VEC, NV, TPG);
    constexpr int kRing = ring_rows(TPG);
    extern __shared__ __align__(16) uint8_t ring_bytes[];  // [kRing][x and z][NV][threads]
    constexpr int kBlk = TPG > 32 ? TPG : kWarpBlock;
    V* ring = reinterpret_cast<V*>(ring_bytes);
    const int slots = gated ? 2 * NV : NV;
    auto ahead = [&](int64_t r, int stage) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + i * TPG;
            const bool live = mine && r < a.rows && j < nvec;
            const uint32_t dst = (uint32_t)__cvta_generic_to_shared(ring + (stage * slots + i) * kBlk + threadIdx.x);
            const int64_t at = live ? (int64_t)j * VEC : 0, rr = live ? r : 0;
            copy_async<sizeof(V)>(dst, x + rr * a.x_stride + at, live);
            if (gated) copy_async<sizeof(V)>(dst + NV * kBlk * sizeof(V), z + rr * a.z_stride + at, live);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int stage = 0;
    if (kUseRing) {
        for (int i = 0; i < kRing; ++i) ahead(row + i * step, i);
    } else {
        load(row);
    }
    // every thread of the block walks as far (blocks larger than a warp meet at barriers)
    for (int64_t r0 = (int64_t)blockIdx.y * rows_per; r0 < a.rows; r0 += step, row += step) {
        float u[NV][VEC];
        V zc[NV];
        float s = 0.f;
        if constexpr (kUseRing) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const V* from = ring + (stage * slots + i) * kBlk + threadIdx.x;
                xr[i] = *from;
                if (gated) zr[i] = from[NV * kBlk];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack<VEC>(xr[i], u[i], (const T*)nullptr);
            zc[i] = zr[i];
            if (before) {
                float gate[VEC];
                unpack<VEC>(zc[i], gate, (const T*)nullptr);
#pragma unroll
                for (int e = 0; e < VEC; ++e) u[i][e] *= silu_f32<T>(gate[e]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += u[i][e];
        }
        if (kUseRing) {
            ahead(row + kRing * step, stage);
            if (++stage == kRing) stage = 0;
        } else if (kKeep) {
            load(row + step);
        }
        float mean = 0.f;
        if (a.flags & MAMBA2_NORM_SUBTRACT_MEAN) mean = group_sum<TPG>(s, smem, turn) / (float)size;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * TPG < nvec) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    u[i][e] -= mean;
                    ss = fmaf(u[i][e], u[i][e], ss);
                }
            }
        }
        const float r = rsqrtf(group_sum<TPG>(ss, smem, turn) / (float)size + a.eps);
        if (mine && row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = lane + i * TPG;
                if (j >= nvec) break;
                float o[VEC];
                if (!kKeep) weights(j, w[0]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = u[i][e] * r * w[kKeep ? i : 0][e];
                if (a.bias) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] += a.bias[c0 + (int64_t)j * VEC + e];
                }
                if (after) {
                    float gate[VEC];
                    unpack<VEC>(zc[i], gate, (const T*)nullptr);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] *= silu_f32<T>(gate[e]);
                } else if (a.flags & MAMBA2_NORM_SILU) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = silu_f32<T>(o[e]);
                }
                *reinterpret_cast<V*>(y + row * a.y_stride + (int64_t)j * VEC) = pack<T, VEC>(o);
            }
        }
        if (!kKeep) load(row + step);
    }
    if (kUseRing) asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int VEC, int NV, int TPG>
cudaError_t launch_n(const NormArgs& a, cudaStream_t st) {
    constexpr int block = TPG > 32 ? TPG : kWarpBlock, per = block / TPG;
    int across = 0;  // as many groups side by side as there are, up to the block
    while ((2 << across) <= per && (1 << across) < a.ngroups) ++across;
    const int64_t gx = (a.ngroups + (1 << across) - 1) >> across, rows_per = per >> across;
    // as many blocks as fit on the GPU at once: each keeps its weights for its share of the rows
    const bool gated = (a.flags & (MAMBA2_NORM_GATE_BEFORE | MAMBA2_NORM_GATE_AFTER)) != 0;
    auto ring_bytes = [](bool z) {
        constexpr int row = NV * block * (int)sizeof(typename VecOf<T, VEC>::type);
        return use_ring<T>(VEC, NV, TPG) ? ring_rows(TPG) * (z ? 2 : 1) * row : 0;
    };
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(k_group_norm<T, VEC, NV, TPG>),
                                                  ring_bytes(true));
    if (e != cudaSuccess) return e;
    auto count = [&](bool z) {
        int n = 0;
        const cudaError_t err =
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_group_norm<T, VEC, NV, TPG>, block, ring_bytes(z));
        return err == cudaSuccess && n > 0 ? n : 1;
    };
    static const int fit[2] = {count(false), count(true)};
    const int resident = fit[gated];
    const int sms = sm_count();
    const int64_t want = (resident * (int64_t)(sms > 0 ? sms : 152) + gx - 1) / gx;
    const int64_t gy = imin64(imin64((a.rows + rows_per - 1) / rows_per, want < 1 ? 1 : want), 65535);
    k_group_norm<T, VEC, NV, TPG><<<dim3((unsigned)gx, (unsigned)gy), block, ring_bytes(gated), st>>>(a, across);
    return cudaGetLastError();
}

// The fewest threads that hold the group.
template <typename T, int VEC>
cudaError_t launch_v(const NormArgs& a, cudaStream_t st) {
    const int64_t n = a.channels / a.ngroups / VEC;
    // single elements: more loads per thread (bf16, gated, us with 8 / 4 / 2: 65536 x 264 in groups of
    // 33 58 / 51 / 80, 16384 x 1028 in groups of 257 86 / 45 / 49, 8192 x 2049 66 / 44 / 50)
    constexpr int K = VEC == 1 ? 4 : 1;
    if (n <= 8 * K) return launch_n<T, VEC, K, 8>(a, st);
    if (n <= 16 * K) return launch_n<T, VEC, K, 16>(a, st);
    if (n <= 32 * K) return launch_n<T, VEC, K, 32>(a, st);
    if (n <= 64 * K) return launch_n<T, VEC, 2 * K, 32>(a, st);
    if (n <= 128 * K) return launch_n<T, VEC, 2 * K, 64>(a, st);
    if (n <= 256 * K) return launch_n<T, VEC, 2 * K, 128>(a, st);
    if (n <= 512 * K) return launch_n<T, VEC, 2 * K, 256>(a, st);
    if (n <= 1024 * K) return launch_n<T, VEC, 2 * K, 512>(a, st);
    if (n <= 2048 * K) return launch_n<T, VEC, 2 * K, 1024>(a, st);
    if (n <= 4096 * K) return launch_n<T, VEC, 4 * K, 1024>(a, st);
    return launch_n<T, VEC, 8 * K, 1024>(a, st);
}

template <typename T>
cudaError_t launch_t(const NormArgs& a, cudaStream_t st) {
    constexpr int VEC = 16 / sizeof(T);
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                        reinterpret_cast<uintptr_t>(a.z);
    auto fits = [&](int n) {
        return (a.channels / a.ngroups) % n == 0 && a.x_stride % n == 0 && a.y_stride % n == 0 && a.z_stride % n == 0 &&
               p % (n * sizeof(T)) == 0;
    };
    if (fits(VEC)) return launch_v<T, VEC>(a, st);
    // (bf16, gated, us in fours / one by one: 16384 x 3200 in groups of 100 99 / 135, 16384 x 2400
    // in groups of 300 81 / 181, 8192 x 2052 in one group 38 / 67)
    if constexpr (VEC == 8)
        if (fits(4)) return launch_v<T, 4>(a, st);
    return launch_v<T, 1>(a, st);
}

}  // namespace

cudaError_t launch_group_norm(const NormArgs& a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace m2
