// api_gated_linear.cu — the extern "C" boundary of include/mamba2_gated_linear.h:
// argument checks and launches.
#include "abi_checks.cuh"
#include "gated_linear.cuh"

using namespace m2;

namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 40;  // of a tensor, strides included
constexpr int64_t kMaxCount = (int64_t)1 << 30;     // tokens, channels
constexpr int64_t kMaxStates = (int64_t)1 << 33;     // of the recurrence: a launch has a block for 32
constexpr size_t kWorkspaceAlign = 256;

bool is_dtype(int32_t d) { return d == MAMBA2_F32 || d == MAMBA2_BF16; }
int elt_bytes(int32_t dtype) { return dtype == MAMBA2_BF16 ? 2 : 4; }

// Every tensor is there and aligned; no output lies over an input or another output (but for those of `same`, which
// may be one tensor: an output's index and an input's, both with one stride).
template <int NI, int NO>
mamba2_status check(const Tensor (&in)[NI], const Tensor (&out)[NO], int same_out = -1, int same_in = -1) {
    auto fits = [](const Tensor& t) {
        if (!t.p) return t.optional || t.rows <= 0 || t.width <= 0;
        return is_aligned(t.p, t.align);
    };
    for (const Tensor& t : in)
        if (!fits(t)) return MAMBA2_ERR_INVALID_ARG;
    for (const Tensor& t : out)
        if (!fits(t)) return MAMBA2_ERR_INVALID_ARG;
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i) {
            if (o == same_out && i == same_in && out[o].p == in[i].p && out[o].stride == in[i].stride) continue;
            if (overlap(out[o], in[i])) return MAMBA2_ERR_INVALID_ARG;
        }
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return MAMBA2_ERR_INVALID_ARG;
    }
    return MAMBA2_OK;
}

// 0 means packed; else at least the row's width.
mamba2_status resolve(int64_t* stride, int64_t width, int64_t rows) {
    if (*stride == 0) *stride = width;
    if (*stride < width) return MAMBA2_ERR_INVALID_ARG;
    if (rows > 0 && *stride > kMaxElements / rows) return MAMBA2_ERR_UNSUPPORTED;
    return MAMBA2_OK;
}
template <int N>
mamba2_status resolve_all(int64_t* const (&strides)[N], int64_t width, int64_t rows) {
    for (int64_t* s : strides) {
        const mamba2_status rc = resolve(s, width, rows);
        if (rc != MAMBA2_OK) return rc;
    }
    return MAMBA2_OK;
}

mamba2_status fill(void* dst, const void* src, int64_t bytes, cudaStream_t st) {
    if (!dst || bytes == 0 || dst == src) return MAMBA2_OK;
    return from_cuda(src ? cudaMemcpyAsync(dst, src, (size_t)bytes, cudaMemcpyDeviceToDevice, st)
                         : cudaMemsetAsync(dst, 0, (size_t)bytes, st));
}

// ------------------------------------------------- gated linear recurrence
mamba2_status check_glr(const mamba2_glr_shape* s) {
    if (!s || !is_dtype(s->dtype) || s->flags != 0) return MAMBA2_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1) return MAMBA2_ERR_INVALID_ARG;
    if (s->batch > 65535 || s->seqlen > kMaxCount || s->channels > kMaxCount) return MAMBA2_ERR_UNSUPPORTED;
    const int64_t rows = s->batch * s->seqlen;
    if (rows > 0 && s->channels > kMaxElements / rows) return MAMBA2_ERR_UNSUPPORTED;
    if (s->batch * s->channels > kMaxStates) return MAMBA2_ERR_UNSUPPORTED;
    return MAMBA2_OK;
}
int64_t chunks_of(const mamba2_glr_shape& s) { return (s.seqlen + MAMBA2_GLR_CHUNK - 1) / MAMBA2_GLR_CHUNK; }

mamba2_status glr(bool step, const mamba2_glr_shape* s, const void* x, const void* r, const void* i, const void* z,
                  const float* A, const int32_t* lengths, const float* init, void* y, float* chunk_states,
                  float* final_state, cudaStream_t st) {
    mamba2_status rc = check_glr(s);
    if (rc != MAMBA2_OK) return rc;
    if (step && s->seqlen != 1) return MAMBA2_ERR_INVALID_ARG;
    const int64_t rows = s->batch * s->seqlen, C = s->channels;
    GlrArgs a;
    a.x_stride = s->x_stride, a.r_stride = s->r_stride, a.i_stride = s->i_stride;
    a.z_stride = s->z_stride, a.y_stride = s->y_stride;
    int64_t* const strides[] = {&a.x_stride, &a.r_stride, &a.i_stride, &a.z_stride, &a.y_stride};
    if ((rc = resolve_all(strides, C, rows)) != MAMBA2_OK) return rc;
    const int e = elt_bytes(s->dtype);
    const int64_t state = s->batch * C * 4;
    const Tensor in[] = {packed(init, state, true),
                         sequence(x, rows, C, a.x_stride, e),
                         sequence(r, rows, C, a.r_stride, e),
                         sequence(i, rows, C, a.i_stride, e),
                         sequence(z, rows, C, a.z_stride, e, true),
                         packed(A, C * 4),
                         packed(lengths, s->batch * 4, true, 4)};
    const Tensor out[] = {packed(final_state, state, !step), sequence(y, rows, C, a.y_stride, e),
                          packed(chunk_states, chunks_of(*s) * state, true)};
    // in place (the step): a thread reads its state before it writes it
    if ((rc = check(in, out, step ? 0 : -1, step ? 0 : -1)) != MAMBA2_OK) return rc;
    if (s->batch == 0) return MAMBA2_OK;
    if (s->seqlen == 0) return fill(final_state, init, state, st);
    a.batch = s->batch, a.seqlen = s->seqlen, a.channels = C;
    a.x = x, a.r = r, a.i = i, a.z = z, a.A = A, a.lengths = lengths, a.init = init;
    a.y = y, a.chunk_states = chunk_states, a.final_state = final_state;
    const bool bf16 = s->dtype == MAMBA2_BF16;
    return from_cuda(step ? launch_glr_step(a, bf16, st) : launch_glr_fwd(a, bf16, st));
}

size_t rounded(int64_t floats) {
    return ((size_t)floats * 4 + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign;
}
bool has_workspace(const void* p, size_t bytes, size_t need) {
    return bytes >= need && (need == 0 || (p && is_aligned(p, (int)kWorkspaceAlign)));
}

// --------------------------------------------- gradient of the convolution
mamba2_status check_conv(const mamba2_conv_shape* s) {
    if (!s || !is_dtype(s->dtype) || (s->flags & ~MAMBA2_CONV_SILU)) return MAMBA2_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->width < 2) return MAMBA2_ERR_INVALID_ARG;
    if (s->width > 8 || s->batch > 65535 || s->seqlen > kMaxCount || s->channels > kMaxCount)
        return MAMBA2_ERR_UNSUPPORTED;
    const int64_t rows = s->batch * s->seqlen;
    if (rows > 0 && s->channels > kMaxElements / rows) return MAMBA2_ERR_UNSUPPORTED;
    return MAMBA2_OK;
}

// ------------------------------------------------------------- block norm
mamba2_status check_norm(const mamba2_block_norm_shape* s) {
    if (!s || !is_dtype(s->dtype) || !is_dtype(s->residual_dtype)) return MAMBA2_ERR_INVALID_ARG;
    if (s->flags & ~(MAMBA2_BLOCK_NORM_POST | MAMBA2_BLOCK_NORM_PRE)) return MAMBA2_ERR_INVALID_ARG;
    if (s->rows < 0 || s->channels < 1 || !(s->eps > 0.f)) return MAMBA2_ERR_INVALID_ARG;
    if (s->channels > 32768 || s->rows >= ((int64_t)1 << 31)) return MAMBA2_ERR_UNSUPPORTED;
    // (a residual in fewer bits than the values that are added to it)
    if (s->dtype == MAMBA2_F32 && s->residual_dtype == MAMBA2_BF16) return MAMBA2_ERR_UNSUPPORTED;
    return MAMBA2_OK;
}

}  // namespace

extern "C" {

mamba2_status mamba2_glr_fwd(const mamba2_glr_shape* shape, const void* x, const void* r, const void* i, const void* z,
                             const float* A, const int32_t* lengths, const float* initial_state, void* y,
                             float* chunk_states, float* final_state, struct CUstream_st* stream) {
    return glr(false, shape, x, r, i, z, A, lengths, initial_state, y, chunk_states, final_state,
               (cudaStream_t)stream);
}

mamba2_status mamba2_glr_step(const mamba2_glr_shape* shape, const void* x, const void* r, const void* i,
                              const void* z, const float* A, const float* state_in, float* state_out, void* y,
                              struct CUstream_st* stream) {
    return glr(true, shape, x, r, i, z, A, nullptr, state_in, y, nullptr, state_out, (cudaStream_t)stream);
}

size_t mamba2_glr_bwd_workspace_size(const mamba2_glr_shape* s) {
    if (check_glr(s) != MAMBA2_OK || s->batch == 0 || s->seqlen == 0) return 0;
    return rounded(s->batch * s->channels);  // each batch row's part of A dA
}

mamba2_status mamba2_glr_bwd(const mamba2_glr_shape* s, const mamba2_glr_grad_strides* grad_strides, const void* dy,
                             const void* x, const void* r, const void* i, const void* z, const float* A,
                             const int32_t* lengths, const float* chunk_states, const float* dfinal_state, void* dx,
                             void* dr, void* di, void* dz, float* dA, float* dinitial_state, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream) {
    mamba2_status rc = check_glr(s);
    if (rc != MAMBA2_OK) return rc;
    const mamba2_glr_grad_strides g = grad_strides ? *grad_strides : mamba2_glr_grad_strides{0, 0, 0, 0};
    const int64_t rows = s->batch * s->seqlen, C = s->channels;
    GlrBwdArgs a;
    a.x_stride = s->x_stride, a.r_stride = s->r_stride, a.i_stride = s->i_stride, a.z_stride = s->z_stride;
    a.dy_stride = s->y_stride, a.dx_stride = g.dx_stride, a.dr_stride = g.dr_stride, a.di_stride = g.di_stride;
    a.dz_stride = g.dz_stride;
    int64_t* const strides[] = {&a.x_stride,  &a.r_stride,  &a.i_stride,  &a.z_stride, &a.dy_stride,
                                &a.dx_stride, &a.dr_stride, &a.di_stride, &a.dz_stride};
    if ((rc = resolve_all(strides, C, rows)) != MAMBA2_OK) return rc;
    if ((z != nullptr) != (dz != nullptr) && rows > 0) return MAMBA2_ERR_INVALID_ARG;
    const size_t need = mamba2_glr_bwd_workspace_size(s);
    if (!has_workspace(workspace, workspace_bytes, need)) return MAMBA2_ERR_INVALID_ARG;
    const int e = elt_bytes(s->dtype);
    const int64_t state = s->batch * C * 4;
    const Tensor in[] = {sequence(dy, rows, C, a.dy_stride, e),
                         sequence(x, rows, C, a.x_stride, e),
                         sequence(r, rows, C, a.r_stride, e),
                         sequence(i, rows, C, a.i_stride, e),
                         sequence(z, rows, C, a.z_stride, e, true),
                         packed(A, C * 4),
                         packed(lengths, s->batch * 4, true, 4),
                         packed(chunk_states, chunks_of(*s) * state),
                         packed(dfinal_state, state, true)};
    const Tensor out[] = {sequence(dx, rows, C, a.dx_stride, e),
                          sequence(dr, rows, C, a.dr_stride, e),
                          sequence(di, rows, C, a.di_stride, e),
                          sequence(dz, rows, C, a.dz_stride, e, true),
                          packed(dA, C * 4),
                          packed(dinitial_state, state, true),
                          packed(workspace, (int64_t)need, true)};
    if ((rc = check(in, out)) != MAMBA2_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if ((rc = fill(dA, nullptr, C * 4, st)) != MAMBA2_OK) return rc;
        return fill(dinitial_state, dfinal_state, state, st);
    }
    a.batch = s->batch, a.seqlen = s->seqlen, a.channels = C;
    a.dy = dy, a.x = x, a.r = r, a.i = i, a.z = z, a.A = A, a.lengths = lengths;
    a.chunk_states = chunk_states, a.dfinal = dfinal_state;
    a.dx = dx, a.dr = dr, a.di = di, a.dz = dz, a.dA = dA, a.dinit = dinitial_state;
    a.partials = static_cast<float*>(workspace);
    return from_cuda(launch_glr_bwd(a, s->dtype == MAMBA2_BF16, st));
}

size_t mamba2_causal_conv_bwd_workspace_size(const mamba2_conv_shape* s) {
    if (check_conv(s) != MAMBA2_OK || s->batch == 0 || s->seqlen == 0) return 0;
    return rounded(conv_bwd_partials(s->batch, s->seqlen, s->channels, (int)s->width));
}

mamba2_status mamba2_causal_conv_bwd(const mamba2_conv_shape* s, int64_t dx_stride, const void* dy, const void* x,
                                     const float* weight, const float* bias, const int32_t* lengths,
                                     const void* initial_state, const void* dfinal_state, void* dx, float* dweight,
                                     float* dbias, void* dinitial_state, void* workspace, size_t workspace_bytes,
                                     struct CUstream_st* stream) {
    mamba2_status rc = check_conv(s);
    if (rc != MAMBA2_OK) return rc;
    const int64_t rows = s->batch * s->seqlen, C = s->channels;
    ConvBwdArgs a;
    a.x_stride = s->x_stride, a.dy_stride = s->y_stride, a.dx_stride = dx_stride;
    int64_t* const strides[] = {&a.x_stride, &a.dy_stride, &a.dx_stride};
    if ((rc = resolve_all(strides, C, rows)) != MAMBA2_OK) return rc;
    const size_t need = mamba2_causal_conv_bwd_workspace_size(s);
    if (!has_workspace(workspace, workspace_bytes, need)) return MAMBA2_ERR_INVALID_ARG;
    const int e = elt_bytes(s->dtype);
    const int64_t state = s->batch * (s->width - 1) * C * e;
    const Tensor in[] = {sequence(dy, rows, C, a.dy_stride, e),
                         sequence(x, rows, C, a.x_stride, e),
                         packed(weight, C * s->width * 4),
                         packed(bias, C * 4, true),
                         packed(lengths, s->batch * 4, true, 4),
                         packed(initial_state, state, true),
                         packed(dfinal_state, state, true)};
    const Tensor out[] = {sequence(dx, rows, C, a.dx_stride, e), packed(dweight, C * s->width * 4),
                          packed(dbias, C * 4, true), packed(dinitial_state, state, true),
                          packed(workspace, (int64_t)need, true)};
    if ((rc = check(in, out)) != MAMBA2_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if ((rc = fill(dweight, nullptr, C * s->width * 4, st)) != MAMBA2_OK) return rc;
        if ((rc = fill(dbias, nullptr, C * 4, st)) != MAMBA2_OK) return rc;
        return fill(dinitial_state, dfinal_state, state, st);
    }
    a.batch = s->batch, a.seqlen = s->seqlen, a.channels = C, a.width = (int)s->width;
    a.dy = dy, a.x = x, a.weight = weight, a.bias = bias, a.lengths = lengths;
    a.init = initial_state, a.dfinal = dfinal_state;
    a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.dinit = dinitial_state;
    a.silu = (s->flags & MAMBA2_CONV_SILU) != 0;
    a.partials = static_cast<float*>(workspace);
    return from_cuda(launch_causal_conv_bwd(a, s->dtype == MAMBA2_BF16, st));
}

mamba2_status mamba2_block_norm_fwd(const mamba2_block_norm_shape* s, const void* x, const void* z,
                                    const void* residual, const float* post_weight, const float* scale,
                                    const float* pre_weight, void* residual_out, void* y,
                                    struct CUstream_st* stream) {
    mamba2_status rc = check_norm(s);
    if (rc != MAMBA2_OK) return rc;
    const int64_t rows = s->rows, C = s->channels;
    BlockNormArgs a;
    a.post = (s->flags & MAMBA2_BLOCK_NORM_POST) != 0, a.pre = (s->flags & MAMBA2_BLOCK_NORM_PRE) != 0;
    a.x_stride = s->x_stride, a.z_stride = s->z_stride, a.res_stride = s->residual_stride;
    a.out_stride = s->residual_out_stride, a.y_stride = s->y_stride;
    int64_t* const strides[] = {&a.x_stride, &a.z_stride, &a.res_stride, &a.out_stride, &a.y_stride};
    if ((rc = resolve_all(strides, C, rows)) != MAMBA2_OK) return rc;
    if ((y != nullptr) != a.pre && rows > 0) return MAMBA2_ERR_INVALID_ARG;
    if ((!a.post && post_weight) || (!a.pre && pre_weight)) return MAMBA2_ERR_INVALID_ARG;
    const int e = elt_bytes(s->dtype), f = elt_bytes(s->residual_dtype);
    const Tensor in[] = {sequence(residual, rows, C, a.res_stride, f, true),
                         sequence(x, rows, C, a.x_stride, e),
                         sequence(z, rows, C, a.z_stride, e, true),
                         packed(post_weight, C * 4, true),
                         packed(scale, C * 4, true),
                         packed(pre_weight, C * 4, true)};
    const Tensor out[] = {sequence(residual_out, rows, C, a.out_stride, f), sequence(y, rows, C, a.y_stride, e, true)};
    // in place: a thread has read its channels of a row before it writes them
    if ((rc = check(in, out, 0, 0)) != MAMBA2_OK) return rc;
    if (rows == 0) return MAMBA2_OK;
    a.rows = rows, a.channels = C, a.eps = s->eps;
    a.x = x, a.z = z, a.res = residual, a.out = residual_out, a.y = y;
    a.post_weight = post_weight, a.scale = scale, a.pre_weight = pre_weight;
    return from_cuda(launch_block_norm(a, s->dtype == MAMBA2_BF16, s->residual_dtype == MAMBA2_BF16,
                                       (cudaStream_t)stream));
}

size_t mamba2_block_norm_bwd_workspace_size(const mamba2_block_norm_shape* s) {
    if (check_norm(s) != MAMBA2_OK || s->rows == 0) return 0;
    return rounded(block_norm_bwd_partials(s->rows, s->channels));
}

mamba2_status mamba2_block_norm_bwd(const mamba2_block_norm_shape* s, const mamba2_block_norm_grad_strides* grad_strides,
                                    const void* dresidual_out, const void* dy, const void* x, const void* z,
                                    const void* residual_out, const float* post_weight, const float* scale,
                                    const float* pre_weight, void* dx, void* dz, void* dresidual, float* dpost_weight,
                                    float* dscale, float* dpre_weight, void* workspace, size_t workspace_bytes,
                                    struct CUstream_st* stream) {
    mamba2_status rc = check_norm(s);
    if (rc != MAMBA2_OK) return rc;
    const mamba2_block_norm_grad_strides g =
        grad_strides ? *grad_strides : mamba2_block_norm_grad_strides{0, 0, 0, 0};
    const int64_t rows = s->rows, C = s->channels;
    BlockNormBwdArgs a;
    a.post = (s->flags & MAMBA2_BLOCK_NORM_POST) != 0, a.pre = (s->flags & MAMBA2_BLOCK_NORM_PRE) != 0;
    a.x_stride = s->x_stride, a.z_stride = s->z_stride, a.out_stride = s->residual_out_stride;
    a.dy_stride = s->y_stride, a.dx_stride = g.dx_stride, a.dz_stride = g.dz_stride;
    a.dout_stride = g.dresidual_out_stride, a.dres_stride = g.dresidual_stride;
    int64_t* const strides[] = {&a.x_stride,  &a.z_stride,  &a.out_stride,  &a.dy_stride,
                                &a.dx_stride, &a.dz_stride, &a.dout_stride, &a.dres_stride};
    if ((rc = resolve_all(strides, C, rows)) != MAMBA2_OK) return rc;
    if (rows > 0 && ((dy != nullptr) != a.pre || (residual_out != nullptr) != a.pre || (z != nullptr) != (dz != nullptr)))
        return MAMBA2_ERR_INVALID_ARG;
    if ((!a.post && (post_weight || dpost_weight)) || (!a.pre && (pre_weight || dpre_weight)))
        return MAMBA2_ERR_INVALID_ARG;
    const size_t need = mamba2_block_norm_bwd_workspace_size(s);
    if (!has_workspace(workspace, workspace_bytes, need)) return MAMBA2_ERR_INVALID_ARG;
    const int e = elt_bytes(s->dtype), f = elt_bytes(s->residual_dtype);
    const Tensor in[] = {sequence(dresidual_out, rows, C, a.dout_stride, f, true),
                         sequence(dy, rows, C, a.dy_stride, e, true),
                         sequence(x, rows, C, a.x_stride, e),
                         sequence(z, rows, C, a.z_stride, e, true),
                         sequence(residual_out, rows, C, a.out_stride, f, true),
                         packed(post_weight, C * 4, true),
                         packed(scale, C * 4, true),
                         packed(pre_weight, C * 4, true)};
    const Tensor out[] = {sequence(dresidual, rows, C, a.dres_stride, f, true),
                          sequence(dx, rows, C, a.dx_stride, e),
                          sequence(dz, rows, C, a.dz_stride, e, true),
                          packed(dpost_weight, C * 4, true),
                          packed(dscale, C * 4, true),
                          packed(dpre_weight, C * 4, true),
                          packed(workspace, (int64_t)need, true)};
    if ((rc = check(in, out, 0, 0)) != MAMBA2_OK) return rc;
    const cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        for (float* w : {dpost_weight, dscale, dpre_weight})
            if ((rc = fill(w, nullptr, C * 4, st)) != MAMBA2_OK) return rc;
        return MAMBA2_OK;
    }
    a.rows = rows, a.channels = C, a.eps = s->eps;
    a.dout = dresidual_out, a.dy = dy, a.x = x, a.z = z, a.out = residual_out;
    a.post_weight = post_weight, a.scale = scale, a.pre_weight = pre_weight;
    a.dx = dx, a.dz = dz, a.dres = dresidual, a.dpost = dpost_weight, a.dscale = dscale, a.dpre = dpre_weight;
    a.partials = static_cast<float*>(workspace);
    return from_cuda(launch_block_norm_bwd(a, s->dtype == MAMBA2_BF16, s->residual_dtype == MAMBA2_BF16, st));
}

}  // extern "C"
