// C entry points of the root-mean-square norm: argument checks, then one of the launch functions.
#include <algorithm>
#include <cmath>

#include "norm.h"

using namespace wtconv;

namespace wtconv {

int norm_backward_grid(int rows, int C) {
    const int threads = C <= 1024 ? 128 : C <= 4096 ? 256 : 512, at_once = C <= 512 ? 4 : 1;  // rows of a CTA
    return std::min(ceil_div(rows, at_once), sm_count() * (C <= 512 ? 8 : 1024 / threads));
}

}  // namespace wtconv

namespace {

int check_shape(const wtconv_rms_shape *s) {
    if (s == nullptr || s->rows <= 0 || s->rows > (1 << 30) || s->C <= 0 || s->C > WTCONV_RMS_MAX_CHANNELS || !(s->eps >= 0.f) ||
        std::isinf(s->eps))
        return WTCONV_ERR_INVALID_ARG;
    return dtype_ok(s->dtype) && (s->total_dtype == s->dtype || s->total_dtype == WTCONV_F32) ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

bool present(const wtconv_rms_tensor *t) { return t != nullptr && t->p != nullptr; }
bool tensor_ok(const wtconv_rms_tensor *t, const wtconv_rms_shape &s, int dtype, bool output) {
    return t != nullptr && activation_ok(t->p, 0, t->row, 1, s.rows, s.C, dtype, output);
}
// Whether rows start at multiples of 16 bytes.
bool wide(const wtconv_rms_tensor &t, const wtconv_rms_shape &s, int dtype) {
    return t.p == nullptr || (aligned_to(t.p, 16) && (s.rows == 1 || t.row * elem_bytes_of(dtype) % 16 == 0));
}

int forward(NormArgs &a, const wtconv_rms_shape *shape, const wtconv_rms_tensor *x, const wtconv_rms_tensor *residual, const float *w,
            const wtconv_rms_tensor *total, wtconv_stream_t stream) {
    const wtconv_rms_shape &s = *shape;
    const bool added = present(residual);
    if (!tensor_ok(x, s, s.dtype, false) || !f32_ok(w, false) ||
        (added && (!tensor_ok(residual, s, s.total_dtype, false) || !tensor_ok(total, s, s.total_dtype, true))) ||
        (!added && s.total_dtype != s.dtype))
        return WTCONV_ERR_INVALID_ARG;
    a.s = s, a.x = *x, a.w = w;
    if (added) a.residual = *residual, a.total = *total;
    const int v = 16 / elem_bytes_of(s.dtype);
    a.wide = s.C % v == 0 && wide(a.x, s, s.dtype) && wide(a.y, s, s.dtype) && wide(a.residual, s, s.total_dtype) &&
             wide(a.total, s, s.total_dtype) && aligned_to(w, 16) && aligned_to(a.q, 16);
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool f32 = s.total_dtype == WTCONV_F32;
    return status_of(s.dtype == WTCONV_F32    ? launch_norm_forward<float, float>(a, st)
                     : s.dtype == WTCONV_BF16 ? (f32 ? launch_norm_forward<__nv_bfloat16, float>(a, st)
                                                     : launch_norm_forward<__nv_bfloat16, __nv_bfloat16>(a, st))
                                              : (f32 ? launch_norm_forward<__half, float>(a, st) : launch_norm_forward<__half, __half>(a, st)));
}

}  // namespace

extern "C" {

int wtconv_rms_forward(const wtconv_rms_shape *shape, const wtconv_rms_tensor *x, const wtconv_rms_tensor *residual, const float *w,
                       const wtconv_rms_tensor *y, const wtconv_rms_tensor *total, float *rstd, wtconv_stream_t stream) {
    const int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    if (!tensor_ok(y, *shape, shape->dtype, true) || !f32_ok(rstd, true)) return WTCONV_ERR_INVALID_ARG;
    NormArgs a = {};
    a.y = *y, a.rstd = rstd;
    return forward(a, shape, x, residual, w, total, stream);
}

int wtconv_rms_forward_e4m3(const wtconv_rms_shape *shape, const wtconv_rms_tensor *x, const wtconv_rms_tensor *residual, const float *w,
                            int block, void *q, float *scales, const wtconv_rms_tensor *total, wtconv_stream_t stream) {
    const int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    if (block != 0 && block != 128) return WTCONV_ERR_UNSUPPORTED;
    if (q == nullptr || !f32_ok(scales, false)) return WTCONV_ERR_INVALID_ARG;
    NormArgs a = {};
    a.q = static_cast<unsigned char *>(q), a.scales = scales, a.block = block, a.blocks = block ? ceil_div(shape->C, block) : 1;
    return forward(a, shape, x, residual, w, total, stream);
}

size_t wtconv_rms_workspace_size(const wtconv_rms_shape *shape) {
    if (check_shape(shape) != WTCONV_OK) return 0;
    return (size_t)norm_backward_grid(shape->rows, shape->C) * shape->C * sizeof(float);
}

int wtconv_rms_backward(const wtconv_rms_shape *shape, const wtconv_rms_tensor *dy, const wtconv_rms_tensor *total, const float *w,
                        const float *rstd, const wtconv_rms_tensor *d_total, const wtconv_rms_tensor *dx,
                        const wtconv_rms_tensor *d_residual, float *dw, void *workspace, size_t workspace_bytes,
                        wtconv_stream_t stream) {
    const int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    const wtconv_rms_shape &s = *shape;
    if (!tensor_ok(dy, s, s.dtype, false) || !tensor_ok(total, s, s.total_dtype, false) || !f32_ok(w, false) || !f32_ok(rstd, false) ||
        (present(d_total) && !tensor_ok(d_total, s, s.total_dtype, false)) || (present(dx) && !tensor_ok(dx, s, s.dtype, true)) ||
        (present(d_residual) && !tensor_ok(d_residual, s, s.total_dtype, true)) || (!present(dx) && !present(d_residual)) ||
        !f32_ok(dw, true))
        return WTCONV_ERR_INVALID_ARG;
    NormArgs a = {};
    a.s = s, a.dy = *dy, a.total = *total, a.w = w, a.rstd_in = rstd, a.dw = dw;
    if (present(d_total)) a.d_total = *d_total;
    if (present(dx)) a.dx = *dx;
    if (present(d_residual)) a.d_residual = *d_residual;
    if (dw != nullptr) {
        if (workspace != nullptr && !aligned_to(workspace, 16)) return WTCONV_ERR_INVALID_ARG;
        if (workspace == nullptr || workspace_bytes < wtconv_rms_workspace_size(shape)) return WTCONV_ERR_WORKSPACE;
        a.part = static_cast<float *>(workspace);
    }
    const int v = 16 / elem_bytes_of(s.dtype);
    a.wide = s.C % v == 0 && wide(a.dy, s, s.dtype) && wide(a.total, s, s.total_dtype) && wide(a.d_total, s, s.total_dtype) &&
             wide(a.dx, s, s.dtype) && wide(a.d_residual, s, s.total_dtype) && aligned_to(w, 16);
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool f32 = s.total_dtype == WTCONV_F32;
    return status_of(s.dtype == WTCONV_F32    ? launch_norm_backward<float, float>(a, st)
                     : s.dtype == WTCONV_BF16 ? (f32 ? launch_norm_backward<__nv_bfloat16, float>(a, st)
                                                     : launch_norm_backward<__nv_bfloat16, __nv_bfloat16>(a, st))
                                              : (f32 ? launch_norm_backward<__half, float>(a, st) : launch_norm_backward<__half, __half>(a, st)));
}

}  // extern "C"
