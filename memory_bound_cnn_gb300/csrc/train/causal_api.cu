// C entry points of the causal convolution: argument checks, then one of the launch functions.
#include <algorithm>

#include "causal.h"

using namespace wtconv;

namespace {

int check_shape(const wtconv_causal_shape *s) {
    if (s == nullptr || s->B <= 0 || s->T <= 0 || s->C <= 0 || (long long)s->B * s->C > 0x7fffffffll || s->T > (1 << 30) ||
        (long long)s->C * 4 > 0x7fffffffll || (s->silu != 0 && s->silu != 1))
        return WTCONV_ERR_INVALID_ARG;
    if (s->layout != WTCONV_SCAN_PLANES && s->layout != WTCONV_SCAN_TOKENS) return WTCONV_ERR_INVALID_ARG;
    return dtype_ok(s->dtype) && s->K >= 2 && s->K <= 4 ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

bool check_tensor(const wtconv_ssm_tensor &t, const wtconv_causal_shape &s, bool output) {
    const bool planes = s.layout == WTCONV_SCAN_PLANES;
    return activation_ok(t.p, t.batch, t.row, s.B, planes ? s.C : s.T, planes ? s.T : s.C, s.dtype, output);
}

bool element_ok(const void *p, const wtconv_causal_shape &s) { return aligned_to(p, elem_bytes_of(s.dtype)); }

// Whether a tensor's rows all start at vectors of n elements.
bool vectors(const wtconv_ssm_tensor &t, const wtconv_causal_shape &s, int n) {
    const bool rows = (s.layout == WTCONV_SCAN_PLANES ? s.C : s.T) > 1;
    return aligned_to(t.p, (size_t)n * elem_bytes_of(s.dtype)) && (!rows || t.row % n == 0) && (s.B == 1 || t.batch % n == 0);
}

// How the work is cut, by the shape alone (the workspace's size has to follow from it).
void plan(CausalArgs &a, bool backward) {
    const wtconv_causal_shape &s = a.s;
    if (s.layout == WTCONV_SCAN_TOKENS) {
        // A strip repeats K-1 positions of its neighbours; shorter ones keep the SMs busy where there is little.
        const long long threads = (long long)s.B * s.C * s.T / 2;
        a.strip = backward ? 128 : 64;
        while (a.strip > 8 && threads / a.strip < (long long)sm_count() * 1024) a.strip /= 2;
        a.strips = ceil_div(s.T, a.strip);
        a.parts = s.B * ceil_div(a.strips, 8);
    } else {
        const int v = backward ? 4 : 16 / elem_bytes_of(s.dtype), n = ceil_div(s.T, v);
        a.row_bits = 0;
        while (a.row_bits < 5 && (1 << a.row_bits) < n) ++a.row_bits;
        // of a row, 8 vectors a lane in one strip
        a.strip = v * 8 << a.row_bits;
        a.strips = ceil_div(s.T, a.strip);
        a.parts = s.B * a.strips;
    }
}

size_t place(CausalArgs &a, void *workspace) {
    float *const p = static_cast<float *>(workspace);
    const size_t w = ((size_t)a.parts * a.s.C * a.s.K + 3) / 4 * 4;
    a.part_w = p, a.part_b = p + w;
    return (w + (size_t)a.parts * a.s.C) * sizeof(float);
}

// Sequences, strips and parts are counted in 31 bits.
bool counts_ok(const CausalArgs &a) { return (long long)a.s.B * a.strips <= 0x7fffffffll; }

template <typename F> cudaError_t by_type(int dtype, F f) {
    return dtype == WTCONV_F32 ? f(0.f) : dtype == WTCONV_BF16 ? f(__nv_bfloat16()) : f(__half());
}

}  // namespace

extern "C" {

size_t wtconv_causal_workspace_size(const wtconv_causal_shape *shape) {
    if (check_shape(shape) != WTCONV_OK) return 0;
    CausalArgs a = {};
    a.s = *shape;
    plan(a, true);
    return counts_ok(a) ? place(a, nullptr) : 0;
}

int wtconv_causal_forward(const wtconv_causal_shape *shape, const wtconv_ssm_tensor *x, const float *w, const float *bias,
                          const void *state, const int *lengths, const wtconv_ssm_tensor *y, void *state_last,
                          wtconv_stream_t stream) {
    const int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    if (x == nullptr || y == nullptr) return WTCONV_ERR_INVALID_ARG;
    CausalArgs a = {};
    a.s = *shape, a.x = *x, a.y = *y, a.w = w, a.bias = bias, a.state = state, a.lengths = lengths, a.state_last = state_last;
    plan(a, false);
    if (!counts_ok(a) || !check_tensor(a.x, a.s, false) || !check_tensor(a.y, a.s, true) || !f32_ok(w, false) || !f32_ok(bias, true) ||
        !element_ok(state, a.s) || !f32_ok(lengths, true) || !element_ok(state_last, a.s))
        return WTCONV_ERR_INVALID_ARG;
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    const int v = planes ? 16 / elem_bytes_of(a.s.dtype) : 2;
    a.wide = vectors(a.x, a.s, v) && vectors(a.y, a.s, v) && (planes || a.s.C % v == 0);
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_type(a.s.dtype, [&](auto t) { return launch_causal_forward<decltype(t)>(a, st); }));
}

int wtconv_causal_backward(const wtconv_causal_shape *shape, const wtconv_ssm_tensor *x, const float *w, const float *bias,
                           const void *state, const int *lengths, const wtconv_ssm_tensor *dy, const void *d_last,
                           const wtconv_ssm_tensor *dx, float *dw, float *d_bias, void *d_state, void *workspace,
                           size_t workspace_bytes, wtconv_stream_t stream) {
    const int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    if (x == nullptr || dy == nullptr || dx == nullptr) return WTCONV_ERR_INVALID_ARG;
    CausalArgs a = {};
    a.s = *shape, a.x = *x, a.dy = *dy, a.dx = *dx, a.w = w, a.bias = bias, a.state = state, a.lengths = lengths;
    a.d_last = d_last, a.dw = dw, a.d_bias = d_bias, a.d_state = d_state;
    plan(a, true);
    if (!counts_ok(a) || !check_tensor(a.x, a.s, false) || !check_tensor(a.dy, a.s, false) || !check_tensor(a.dx, a.s, true) ||
        !f32_ok(w, false) || !f32_ok(bias, true) || !element_ok(state, a.s) || !f32_ok(lengths, true) || !element_ok(d_last, a.s) ||
        !f32_ok(dw, false) || !f32_ok(d_bias, true) || !element_ok(d_state, a.s))
        return WTCONV_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned_to(workspace, 16)) return WTCONV_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < place(a, workspace)) return WTCONV_ERR_WORKSPACE;
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    const int v = planes ? 4 : 2;
    a.wide = vectors(a.x, a.s, v) && vectors(a.dy, a.s, v) && vectors(a.dx, a.s, v) && (planes || a.s.C % v == 0);
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_type(a.s.dtype, [&](auto t) { return launch_causal_backward<decltype(t)>(a, st); }));
}

int wtconv_causal_step(const wtconv_causal_shape *shape, const wtconv_ssm_tensor *x, const float *w, const float *bias, void *pool,
                       int n_states, const int *slots, const wtconv_ssm_tensor *y, wtconv_stream_t stream) {
    if (shape == nullptr || x == nullptr || y == nullptr) return WTCONV_ERR_INVALID_ARG;
    CausalArgs a = {};
    a.s = *shape, a.s.T = 1, a.s.layout = WTCONV_SCAN_TOKENS;
    const int rc = check_shape(&a.s);
    if (rc != WTCONV_OK) return rc;
    a.x = {x->p, x->row, x->row}, a.y = {y->p, y->row, y->row}, a.w = w, a.bias = bias;  // the rows are the batch's
    if (!check_tensor(a.x, a.s, false) || !check_tensor(a.y, a.s, true) || !f32_ok(w, false) || !f32_ok(bias, true) ||
        pool == nullptr || !element_ok(pool, a.s) || !f32_ok(slots, true) || n_states <= 0 || (slots == nullptr && n_states < a.s.B))
        return WTCONV_ERR_INVALID_ARG;
    if ((long long)a.s.B * ceil_div(a.s.C, 128) > 0x7fffffffll) return WTCONV_ERR_INVALID_ARG;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_type(a.s.dtype, [&](auto t) { return launch_causal_step<decltype(t)>(a, pool, n_states, slots, st); }));
}

}  // extern "C"
