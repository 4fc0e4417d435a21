// C entry points of the selective scan: argument checks, then one of the launch functions.
#include "selective.h"

#include <algorithm>

using namespace wtconv;

namespace {

int check_shape(const wtconv_selective_shape *s) {
    if (s == nullptr || s->B <= 0 || s->T <= 0 || s->C <= 0 || s->N <= 0 || s->G <= 0 || s->C % s->G != 0 ||
        s->N > WTCONV_SELECTIVE_MAX_STATES || (long long)s->B * s->C > 0x7fffffffll || s->T > (1 << 30) ||
        (long long)s->C * s->N > 0x7fffffffll || (s->softplus != 0 && s->softplus != 1))
        return WTCONV_ERR_INVALID_ARG;
    if (s->layout != WTCONV_SCAN_PLANES && s->layout != WTCONV_SCAN_TOKENS) return WTCONV_ERR_INVALID_ARG;
    return dtype_ok(s->dtype) ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

// width: C, or G * N
bool check_tensor(const wtconv_ssm_tensor &t, const wtconv_selective_shape &s, int width, bool output) {
    const bool planes = s.layout == WTCONV_SCAN_PLANES;
    return activation_ok(t.p, t.batch, t.row, s.B, planes ? width : s.T, planes ? s.T : width, s.dtype, output);
}

bool inputs_ok(const SelectiveArgs &a) {
    const wtconv_selective_inputs &in = a.in;
    return check_tensor(in.x, a.s, a.s.C, false) && check_tensor(in.dt, a.s, a.s.C, false) &&
           check_tensor(in.Bm, a.s, a.s.G * a.s.N, false) && check_tensor(in.Cm, a.s, a.s.G * a.s.N, false) &&
           (in.z.p == nullptr || check_tensor(in.z, a.s, a.s.C, false)) && f32_ok(in.A, false) && f32_ok(in.D, true) &&
           f32_ok(in.dt_bias, true) && f32_ok(in.h0, true) && f32_ok(in.lengths, true);
}

// Whether pairs of neighbours along the contiguous axis lie at multiples of their size.
bool pairs(const wtconv_ssm_tensor &t, const wtconv_selective_shape &s) {
    // (a row's stride counts with one channel too: B and C have a row to a state)
    return t.p == nullptr || (aligned_to(t.p, 2 * elem_bytes_of(s.dtype)) && t.row % 2 == 0 && (s.B == 1 || t.batch % 2 == 0));
}
// (a group's first channel has to be even too, where channels are neighbours; its first state is where pairs of
// states are read at once, as their number is then a multiple of 8)
bool pairs(const SelectiveArgs &a) {
    if (a.s.layout == WTCONV_SCAN_TOKENS && a.s.G > 1 && a.channels % 2 != 0) return false;
    for (const wtconv_ssm_tensor *t : {&a.in.x, &a.in.dt, &a.in.Bm, &a.in.Cm, &a.in.z, &a.y, &a.dy, &a.g.dx, &a.g.d_dt, &a.g.dz})
        if (!pairs(*t, a.s)) return false;
    return true;
}

// Parts that a sequence is cut into.  Cutting fills the GPU where sequences and tiles of channels are few, or their
// number leaves a last round of CTAs small; it costs a pass of its own (over x, dt and B in the forward, about half of
// the work, over dy, dt, z and C in the backward, a fifth, and two fifths with few states) and the composition of the parts before a CTA's own.
// Time is counted in rounds of 32 positions of a CTA that has an SM for itself: two that share one take 1.3
// times as long, three 1.6, and more wait; a part's first and last
// rounds add some (ends).  (8 x 4096 x 1024 tokens with 16 states, 256 CTAs: forward 236 us in one part, 308
// in two, the backward of that time 906 and 1032; 65,536 pixels of 64 channels, 2 CTAs: 62 us in 76 parts, 52 in the 147 that this gives.)
void plan(int op, SelectiveArgs &a) {
    const bool forward = op == WTCONV_SCAN_OP_FORWARD;
    const int sms = sm_count(), rounds = ceil_div(a.s.T, kSelRound), most = std::max(1, std::min(rounds / 2, 256));
    const int resident = a.lanes == 2 ? (forward ? 3 : 2) : a.lanes == 4 ? 2 : 1;
    const double share[4] = {1, 1, 1.3, 1.6}, pass = forward ? 1.5 : a.lanes == 2 ? 1.4 : 1.2, start = forward ? 4 : 1, join = forward ? 0.05 : 0.02, ends = forward ? 0.5 : 1.5;
    double best = 0;
    for (int parts = 1; parts <= most; ++parts) {
        const int per = ceil_div(rounds, parts), used = ceil_div(rounds, per);
        if (used > 1 && (long long)a.ctas() * used > 0x7fffffffll) break;
        const long long on_sm = ((long long)a.ctas() * used + sms - 1) / sms;
        const double load = on_sm <= resident ? share[on_sm] : on_sm * share[resident] / resident;
        const double time = (per + ends) * load * (used > 1 ? pass : 1) + (used > 1 ? start + join * used : 0);
        if (parts > 1 && time >= best) continue;
        best = time, a.segment = per * kSelRound, a.segments = used;
    }
    if (a.segments == 1) a.segment = a.s.T;
}

SelectiveArgs args_of(const wtconv_selective_shape &s) {
    SelectiveArgs a = {};
    a.s = s;
    a.channels = s.C / s.G, a.tiles = ceil_div(a.channels, kSelTile);
    a.lanes = selective_lanes(s.N), a.padded = 4 * a.lanes, a.keep = ceil_div(s.T, kSelKeep);
    return a;
}

// Places the workspace's parts (from a null pointer: only their size).
size_t place(int op, SelectiveArgs &a, void *workspace) {
    size_t floats = 0;
    const auto take = [&](size_t n) {
        float *const p = static_cast<float *>(workspace) + floats;
        floats += (n + 3) / 4 * 4;
        return p;
    };
    const size_t parts = (size_t)a.s.B * a.segments * a.s.C;
    if (a.segments > 1) a.ends = take(parts * a.padded), a.steps = take(parts);
    if (op == WTCONV_SCAN_OP_BACKWARD) {
        a.part_bc = take((size_t)a.s.G * a.tiles * a.s.B * a.s.T * 2 * a.padded);
        a.part_a = take(parts * a.s.N), a.part_c = take(2 * parts);
    }
    return floats * sizeof(float);
}

int check_workspace(size_t need, const void *workspace, size_t bytes) {
    if (need == 0) return WTCONV_OK;
    if (workspace != nullptr && !aligned_to(workspace, 16)) return WTCONV_ERR_INVALID_ARG;
    return workspace == nullptr || bytes < need ? WTCONV_ERR_WORKSPACE : WTCONV_OK;
}

// The backward's last sums take a CTA for 32 positions of a group; a grid has at most 2^31 - 1.
bool grid_ok(int op, const wtconv_selective_shape &s) {
    return op == WTCONV_SCAN_OP_FORWARD || (long long)s.B * s.G <= 0x7fffffffll / ceil_div(s.T, kSelRound);
}

template <typename F> cudaError_t by_type(int dtype, F f) {
    return dtype == WTCONV_F32 ? f(0.f) : dtype == WTCONV_BF16 ? f(__nv_bfloat16()) : f(__half());
}

}  // namespace

extern "C" {

size_t wtconv_selective_states_size(const wtconv_selective_shape *shape) {
    if (check_shape(shape) != WTCONV_OK) return 0;
    const SelectiveArgs a = args_of(*shape);
    return (size_t)a.s.B * a.keep * a.s.C * a.padded;
}

size_t wtconv_selective_workspace_size(int op, const wtconv_selective_shape *shape) {
    if (check_shape(shape) != WTCONV_OK || (op != WTCONV_SCAN_OP_FORWARD && op != WTCONV_SCAN_OP_BACKWARD)) return 0;
    if (!grid_ok(op, *shape)) return 0;
    SelectiveArgs a = args_of(*shape);
    plan(op, a);
    return place(op, a, nullptr);
}

int wtconv_selective_forward(const wtconv_selective_shape *shape, const wtconv_selective_inputs *in, const wtconv_ssm_tensor *y,
                             float *h_last, float *states, void *workspace, size_t workspace_bytes, wtconv_stream_t stream) {
    int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    if (in == nullptr || y == nullptr) return WTCONV_ERR_INVALID_ARG;
    SelectiveArgs a = args_of(*shape);
    a.in = *in, a.y = *y, a.h_last = h_last, a.states_out = states;
    if (!inputs_ok(a) || !check_tensor(a.y, a.s, a.s.C, true) || !f32_ok(h_last, true) || !aligned_to(states, 16))
        return WTCONV_ERR_INVALID_ARG;
    a.wide = pairs(a);
    plan(WTCONV_SCAN_OP_FORWARD, a);
    const size_t need = place(WTCONV_SCAN_OP_FORWARD, a, workspace);
    if ((rc = check_workspace(need, workspace, workspace_bytes)) != WTCONV_OK) return rc;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_type(a.s.dtype, [&](auto t) { return launch_selective_forward<decltype(t)>(a, st); }));
}

int wtconv_selective_backward(const wtconv_selective_shape *shape, const wtconv_selective_inputs *in, const float *states,
                              const wtconv_ssm_tensor *dy, const float *dh_last, const wtconv_selective_grads *grads,
                              void *workspace, size_t workspace_bytes, wtconv_stream_t stream) {
    int rc = check_shape(shape);
    if (rc != WTCONV_OK) return rc;
    if (in == nullptr || dy == nullptr || grads == nullptr) return WTCONV_ERR_INVALID_ARG;
    SelectiveArgs a = args_of(*shape);
    a.in = *in, a.dy = *dy, a.states_in = states, a.dh_last = dh_last, a.g = *grads;
    const int width = a.s.G * a.s.N;
    if (!grid_ok(WTCONV_SCAN_OP_BACKWARD, a.s) || !inputs_ok(a) || !check_tensor(a.dy, a.s, a.s.C, false) || !check_tensor(a.g.dx, a.s, a.s.C, true) ||
        !check_tensor(a.g.d_dt, a.s, a.s.C, true) || !check_tensor(a.g.dB, a.s, width, true) ||
        !check_tensor(a.g.dC, a.s, width, true) || (a.in.z.p != nullptr && !check_tensor(a.g.dz, a.s, a.s.C, true)) ||
        states == nullptr || !aligned_to(states, 16) || !f32_ok(dh_last, true) || !f32_ok(a.g.dA, false) || !f32_ok(a.g.dD, true) ||
        !f32_ok(a.g.d_dt_bias, true) || !f32_ok(a.g.d_h0, true))
        return WTCONV_ERR_INVALID_ARG;
    if (a.in.D == nullptr) a.g.dD = nullptr;
    if (a.in.dt_bias == nullptr) a.g.d_dt_bias = nullptr;
    if (a.in.z.p == nullptr) a.g.dz = {};
    a.wide = pairs(a);
    plan(WTCONV_SCAN_OP_BACKWARD, a);
    const size_t need = place(WTCONV_SCAN_OP_BACKWARD, a, workspace);
    if ((rc = check_workspace(need, workspace, workspace_bytes)) != WTCONV_OK) return rc;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_type(a.s.dtype, [&](auto t) { return launch_selective_backward<decltype(t)>(a, st); }));
}

int wtconv_selective_step(const wtconv_selective_shape *shape, const wtconv_selective_inputs *in, float *pool, int n_states,
                          const int *slots, const wtconv_ssm_tensor *y, wtconv_stream_t stream) {
    if (shape == nullptr || in == nullptr || y == nullptr) return WTCONV_ERR_INVALID_ARG;
    wtconv_selective_shape s = *shape;
    s.T = 1, s.layout = WTCONV_SCAN_TOKENS;
    const int rc = check_shape(&s);
    if (rc != WTCONV_OK) return rc;
    SelectiveArgs a = args_of(s);
    a.in = *in, a.y = *y;
    // one position: the rows are the batch's
    for (wtconv_ssm_tensor *t : {&a.in.x, &a.in.dt, &a.in.Bm, &a.in.Cm, &a.in.z, &a.y}) t->batch = t->row;
    if (!inputs_ok(a) || !check_tensor(a.y, a.s, a.s.C, true) || !f32_ok(pool, false) || !f32_ok(slots, true) ||
        n_states <= 0 || (slots == nullptr && n_states < s.B))
        return WTCONV_ERR_INVALID_ARG;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_type(s.dtype, [&](auto t) { return launch_selective_step<decltype(t)>(a, pool, n_states, slots, st); }));
}

}  // extern "C"
