// k_sum_rows.cu — sums over the rows of a matrix of partial sums, the last step of
// the gradients of weights.  Eight threads take every eighth row of a column each.
// It is launched while the kernel that writes the matrix runs, and waits for its end.
#include "gated_linear.cuh"
#include "tc_ptx.cuh"

namespace m2 {
namespace {

constexpr int kCols = 32, kGroups = 8;

__global__ void __launch_bounds__(kCols * kGroups)
k_sum_rows(const float* partials, int64_t rows, int64_t cols, SumOut o0, SumOut o1, SumOut o2, const float* by) {
    __shared__ float part[kGroups][kCols];
    const int x = threadIdx.x % kCols, g = threadIdx.x / kCols;
    const int64_t c = (int64_t)blockIdx.x * kCols + x;
    float s = 0.f;
    tc::griddep_wait();
    if (c < cols) {
#pragma unroll 8
        for (int64_t k = g; k < rows; k += kGroups) s += partials[k * cols + c];
    }
    part[g][x] = s;
    __syncthreads();
    if (g != 0 || c >= cols) return;
#pragma unroll
    for (int q = 1; q < kGroups; ++q) s += part[q][x];
    const int64_t c1 = c - o0.len, c2 = c1 - o1.len;
    if (c1 < 0) {
        if (o0.out) o0.out[c] = by ? s / by[c] : s;
    } else if (c2 < 0) {
        if (o1.out) o1.out[c1] = s;
    } else if (o2.out) {
        o2.out[c2] = s;
    }
}

}  // namespace

cudaError_t launch_sum_rows(const float* partials, int64_t rows, SumOut o0, SumOut o1, SumOut o2, const float* by,
                            cudaStream_t st) {
    const int64_t cols = o0.len + o1.len + o2.len;
    if (cols == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cols + kCols - 1) / kCols));
    cfg.blockDim = dim3(kCols * kGroups);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, k_sum_rows, partials, rows, cols, o0, o1, o2, by);
    return launched == cudaSuccess ? cudaGetLastError() : (cudaGetLastError(), launched);
}

}  // namespace m2
