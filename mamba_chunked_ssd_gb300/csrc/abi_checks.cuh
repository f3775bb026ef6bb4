// abi_checks.cuh — argument checks shared by the extern "C" entry points: tensor
// pointers are present and aligned, and no output overlaps an input or another
// output, where both may be runs of elements side by side in rows of a wider tensor.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mamba2_ssd.h"

namespace m2 {

// Checks of a mamba2_shape that every entry point makes (api.cu).
mamba2_status check_shape(const mamba2_shape* s);

struct Range {
    uintptr_t lo, hi;
};
inline Range range_of(const void* p, int64_t bytes) {
    return {reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes};
}
inline bool overlap(Range a, Range b) { return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi; }

// A tensor argument: pointer, byte size, whether it may be null, alignment.
struct Arg {
    const void* p;
    int64_t bytes;
    bool optional;
    int align = 16;
};

inline bool is_aligned(const void* p, int align) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(align - 1)) == 0;
}

inline mamba2_status check_ptrs(const Arg* in, int nin, const Arg* out, int nout) {
    for (int i = 0; i < nin + nout; ++i) {
        const Arg& a = i < nin ? in[i] : out[i - nin];
        if (!a.p) {
            if (!a.optional && a.bytes > 0) return MAMBA2_ERR_INVALID_ARG;
            continue;
        }
        if (!is_aligned(a.p, a.align)) return MAMBA2_ERR_INVALID_ARG;
    }
    for (int o = 0; o < nout; ++o) {
        if (!out[o].p) continue;
        const Range ro = range_of(out[o].p, out[o].bytes);
        for (int i = 0; i < nin; ++i)
            if (in[i].p && overlap(ro, range_of(in[i].p, in[i].bytes))) return MAMBA2_ERR_INVALID_ARG;
        for (int j = o + 1; j < nout; ++j)
            if (out[j].p && overlap(ro, range_of(out[j].p, out[j].bytes))) return MAMBA2_ERR_INVALID_ARG;
    }
    return MAMBA2_OK;
}

// A tensor argument: `rows` runs of `width` bytes, `stride` bytes from start to start.
struct Tensor {
    const void* p;
    int64_t rows, width, stride;
    bool optional;
    int align;
};
inline Tensor sequence(const void* p, int64_t rows, int64_t channels, int64_t stride, int e, bool optional = false) {
    return {p, rows, channels * e, stride * e, optional, e};
}
inline Tensor packed(const void* p, int64_t bytes, bool optional = false, int align = 16) {
    return {p, bytes > 0, bytes, bytes, optional, align};
}

inline bool overlap(const Tensor& a, const Tensor& b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const Range ra = range_of(a.p, (a.rows - 1) * a.stride + a.width),
                rb = range_of(b.p, (b.rows - 1) * b.stride + b.width);
    if (!overlap(ra, rb)) return false;
    if (a.stride != b.stride || a.rows < 2 || b.rows < 2) return true;
    // one stride: b's runs lie at one place between a's, or over them
    const int64_t s = a.stride;
    const int64_t d = rb.lo >= ra.lo ? (int64_t)((rb.lo - ra.lo) % (uint64_t)s)
                                     : (s - (int64_t)((ra.lo - rb.lo) % (uint64_t)s)) % s;
    return d < a.width || d + b.width > s;
}

inline mamba2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MAMBA2_OK : MAMBA2_ERR_CUDA; }

}  // namespace m2
