// api_gated_delta.cu — the extern "C" boundary of include/mamba2_gated_delta.h:
// argument checks and launches.
#include "abi_checks.cuh"
#include "gated_delta.cuh"
#include "mamba2_gated_delta.h"

using namespace m2;

namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 40;  // of a tensor, strides included

int elt_bytes(int32_t dtype) { return dtype == MAMBA2_BF16 ? 2 : 4; }

// Bytes from the first to the last element of `rows` rows of `width` elements.
int64_t span_bytes(int64_t rows, int64_t stride, int64_t width, int e) {
    return rows > 0 ? ((rows - 1) * stride + width) * e : 0;
}

// 0 means packed; else at least the row's width.
mamba2_status resolve_stride(int64_t* stride, int64_t width, int64_t rows) {
    if (*stride == 0) *stride = width;
    if (*stride < width) return MAMBA2_ERR_INVALID_ARG;
    if (rows > 0 && *stride > kMaxElements / rows) return MAMBA2_ERR_UNSUPPORTED;
    return MAMBA2_OK;
}

// final_state <- initial_state (or zeros) where there is no token.
mamba2_status copy_state(void* dst, const void* src, int64_t bytes, cudaStream_t st) {
    if (!dst || dst == src || bytes == 0) return MAMBA2_OK;
    return from_cuda(src ? cudaMemcpyAsync(dst, src, (size_t)bytes, cudaMemcpyDeviceToDevice, st)
                         : cudaMemsetAsync(dst, 0, (size_t)bytes, st));
}

mamba2_status gdr(bool step, const mamba2_shape* shape, const mamba2_gdr_options* o, const void* q, const void* k,
                  const void* v, const float* gate, const float* beta, const int32_t* lengths, const float* init,
                  void* y, float* final_state, cudaStream_t st) {
    mamba2_status rc = check_shape(shape);
    if (rc != MAMBA2_OK) return rc;
    if (!o || o->reserved != 0 || (o->flags & ~MAMBA2_GDR_QK_L2NORM)) return MAMBA2_ERR_INVALID_ARG;
    const bool l2norm = (o->flags & MAMBA2_GDR_QK_L2NORM) != 0;
    if (l2norm && !(o->l2_eps > 0.f)) return MAMBA2_ERR_INVALID_ARG;
    if (step && shape->seqlen != 1) return MAMBA2_ERR_INVALID_ARG;
    const int64_t rows = shape->batch * shape->seqlen;
    const int64_t wqk = shape->ngroups * shape->dstate, wv = shape->nheads * shape->headdim;
    GdrArgs a;
    a.q_stride = o->q_stride, a.k_stride = o->k_stride, a.v_stride = o->v_stride;
    if ((rc = resolve_stride(&a.q_stride, wqk, rows)) != MAMBA2_OK) return rc;
    if ((rc = resolve_stride(&a.k_stride, wqk, rows)) != MAMBA2_OK) return rc;
    if ((rc = resolve_stride(&a.v_stride, wv, rows)) != MAMBA2_OK) return rc;
    const int e = elt_bytes(shape->dtype);
    const int64_t gates = rows * shape->nheads * 4;
    const int64_t state = shape->batch * shape->nheads * shape->dstate * shape->headdim * 4;
    // In place (step only): each state element is read and then written by
    // the same thread.
    const bool in_place = step && init != nullptr && init == final_state;
    const Arg in[] = {{q, span_bytes(rows, a.q_stride, wqk, e), false, e},
                      {k, span_bytes(rows, a.k_stride, wqk, e), false, e},
                      {v, span_bytes(rows, a.v_stride, wv, e), false, e},
                      {gate, gates, false},
                      {beta, gates, false},
                      {lengths, shape->batch * 4, true, 4},
                      {in_place ? nullptr : init, state, true}};
    const Arg out[] = {{y, rows * wv * e, false}, {final_state, state, !step}};
    if ((rc = check_ptrs(in, 7, out, 2)) != MAMBA2_OK) return rc;
    if (shape->batch == 0) return MAMBA2_OK;
    if (shape->seqlen == 0) return copy_state(final_state, init, state, st);
    a.g = make_geom(*shape);
    a.q = q, a.k = k, a.v = v, a.gate = gate, a.beta = beta, a.lengths = lengths;
    a.init = init, a.y = y, a.final_state = final_state;
    a.scale = o->scale, a.l2_eps = o->l2_eps, a.l2norm = l2norm;
    const bool bf16 = shape->dtype == MAMBA2_BF16;
    return from_cuda(step ? launch_gdr_step(a, bf16, st) : launch_gdr_fwd(a, bf16, st));
}

mamba2_status conv(bool step, const mamba2_conv_shape* s, const void* x, const float* weight, const float* bias,
                   const int32_t* lengths, const void* init, void* y, void* final_state, cudaStream_t st) {
    if (!s || (s->dtype != MAMBA2_F32 && s->dtype != MAMBA2_BF16) || (s->flags & ~MAMBA2_CONV_SILU))
        return MAMBA2_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->width < 2) return MAMBA2_ERR_INVALID_ARG;
    if (step && s->seqlen != 1) return MAMBA2_ERR_INVALID_ARG;
    if (s->width > 8 || s->batch > 65535 || s->seqlen > ((int64_t)1 << 30) || s->channels > ((int64_t)1 << 30))
        return MAMBA2_ERR_UNSUPPORTED;
    const int64_t rows = s->batch * s->seqlen;
    ConvArgs a;
    a.x_stride = s->x_stride, a.y_stride = s->y_stride;
    mamba2_status rc = resolve_stride(&a.x_stride, s->channels, rows);
    if (rc != MAMBA2_OK) return rc;
    if ((rc = resolve_stride(&a.y_stride, s->channels, rows)) != MAMBA2_OK) return rc;
    const int e = elt_bytes(s->dtype);
    const int64_t state = s->batch * (s->width - 1) * s->channels * e;
    const bool in_place = step && init != nullptr && init == final_state;
    const Arg in[] = {{x, span_bytes(rows, a.x_stride, s->channels, e), false, e},
                      {weight, s->channels * s->width * 4, false},
                      {bias, s->channels * 4, true},
                      {lengths, s->batch * 4, true, 4},
                      {in_place ? nullptr : init, state, true}};
    const Arg out[] = {{y, span_bytes(rows, a.y_stride, s->channels, e), false, e}, {final_state, state, !step}};
    if ((rc = check_ptrs(in, 5, out, 2)) != MAMBA2_OK) return rc;
    if (s->batch == 0) return MAMBA2_OK;
    if (s->seqlen == 0) return copy_state(final_state, init, state, st);
    a.batch = s->batch, a.seqlen = s->seqlen, a.channels = s->channels, a.width = (int)s->width;
    a.x = x, a.weight = weight, a.bias = bias, a.lengths = lengths, a.init = init;
    a.y = y, a.final_state = final_state, a.silu = (s->flags & MAMBA2_CONV_SILU) != 0;
    const bool bf16 = s->dtype == MAMBA2_BF16;
    return from_cuda(step ? launch_causal_conv_step(a, bf16, st) : launch_causal_conv(a, bf16, st));
}

}  // namespace

extern "C" {

mamba2_status mamba2_gdr_fwd(const mamba2_shape* shape, const mamba2_gdr_options* options, const void* q,
                             const void* k, const void* v, const float* g, const float* beta,
                             const int32_t* lengths, const float* initial_state, void* y, float* final_state,
                             struct CUstream_st* stream) {
    return gdr(false, shape, options, q, k, v, g, beta, lengths, initial_state, y, final_state,
               (cudaStream_t)stream);
}

mamba2_status mamba2_gdr_step(const mamba2_shape* shape, const mamba2_gdr_options* options, const void* q,
                              const void* k, const void* v, const float* g, const float* beta,
                              const float* state_in, float* state_out, void* y, struct CUstream_st* stream) {
    return gdr(true, shape, options, q, k, v, g, beta, nullptr, state_in, y, state_out, (cudaStream_t)stream);
}

mamba2_status mamba2_causal_conv_fwd(const mamba2_conv_shape* shape, const void* x, const float* weight,
                                     const float* bias, const int32_t* lengths, const void* initial_state, void* y,
                                     void* final_state, struct CUstream_st* stream) {
    return conv(false, shape, x, weight, bias, lengths, initial_state, y, final_state, (cudaStream_t)stream);
}

mamba2_status mamba2_causal_conv_step(const mamba2_conv_shape* shape, const void* x, const float* weight,
                                      const float* bias, const void* state_in, void* state_out, void* y,
                                      struct CUstream_st* stream) {
    return conv(true, shape, x, weight, bias, nullptr, state_in, y, state_out, (cudaStream_t)stream);
}

mamba2_status mamba2_group_norm(const mamba2_norm_shape* s, const void* x, const void* z, const float* weight,
                                const float* bias, void* y, struct CUstream_st* stream) {
    constexpr int kModes = MAMBA2_NORM_GATE_BEFORE | MAMBA2_NORM_GATE_AFTER | MAMBA2_NORM_SILU;
    if (!s || (s->dtype != MAMBA2_F32 && s->dtype != MAMBA2_BF16) || s->reserved != 0) return MAMBA2_ERR_INVALID_ARG;
    if (s->flags & ~(kModes | MAMBA2_NORM_SUBTRACT_MEAN)) return MAMBA2_ERR_INVALID_ARG;
    const int mode = s->flags & kModes;
    if (mode & (mode - 1)) return MAMBA2_ERR_INVALID_ARG;
    const bool gated = mode == MAMBA2_NORM_GATE_BEFORE || mode == MAMBA2_NORM_GATE_AFTER;
    if (s->rows < 0 || s->channels < 1 || s->ngroups < 1 || s->channels % s->ngroups != 0 || !(s->eps > 0.f))
        return MAMBA2_ERR_INVALID_ARG;
    if (gated != (z != nullptr) && s->rows > 0) return MAMBA2_ERR_INVALID_ARG;
    if (s->channels / s->ngroups > 32768 || s->rows > kMaxElements / s->channels ||
        s->rows * s->ngroups >= ((int64_t)1 << 31))
        return MAMBA2_ERR_UNSUPPORTED;
    NormArgs a;
    a.x_stride = s->x_stride, a.z_stride = s->z_stride, a.y_stride = s->y_stride;
    mamba2_status rc = resolve_stride(&a.x_stride, s->channels, s->rows);
    if (rc != MAMBA2_OK) return rc;
    if ((rc = resolve_stride(&a.z_stride, s->channels, s->rows)) != MAMBA2_OK) return rc;
    if ((rc = resolve_stride(&a.y_stride, s->channels, s->rows)) != MAMBA2_OK) return rc;
    const int e = elt_bytes(s->dtype);
    const Arg in[] = {{x, span_bytes(s->rows, a.x_stride, s->channels, e), false, e},
                      {z, span_bytes(s->rows, a.z_stride, s->channels, e), !gated, e},
                      {weight, s->channels * 4, true},
                      {bias, s->channels * 4, true}};
    const Arg out[] = {{y, span_bytes(s->rows, a.y_stride, s->channels, e), false, e}};
    if ((rc = check_ptrs(in, 4, out, 1)) != MAMBA2_OK) return rc;
    if (s->rows == 0) return MAMBA2_OK;
    a.rows = s->rows, a.channels = s->channels, a.ngroups = s->ngroups;
    a.x = x, a.z = z, a.weight = weight, a.bias = bias, a.y = y, a.eps = s->eps, a.flags = s->flags;
    return from_cuda(launch_group_norm(a, s->dtype == MAMBA2_BF16, (cudaStream_t)stream));
}

}  // extern "C"
