// Python binding of the selective scan, the causal convolution (include/wtconv_ssm.h) and the root-mean-square norm
// (include/wtconv_norm.h).
#include <vector>

#include "common.h"
#include "wtconv_norm.h"
#include "wtconv_ssm.h"

using namespace binding;

namespace {

using Given = optional<Tensor>;

wtconv_ssm_tensor ssm(const Act &a) { return {a.p, (long long)a.batch, (long long)a.row}; }
wtconv_ssm_tensor ssm_activation(const Given &t, const char *name, bool planes, const Tensor &like) {
    return t.has_value() ? ssm(activation(*t, name, planes, &like)) : wtconv_ssm_tensor{};
}

// A contiguous tensor of x's type, or none.
void *like_array(const Given &t, const char *name, c10::IntArrayRef shape, const Tensor &x) {
    if (!t.has_value()) return nullptr;
    if (t->device() != x.device() || t->scalar_type() != x.scalar_type() || t->sizes() != shape || !t->is_contiguous())
        refuse(std::string(name) + " must be a contiguous tensor of x's dtype and of shape " + text(shape) + " on " + x.device().str());
    return t->data_ptr();
}

// ------------------------------------------------------------------------------------ selective scan

// What the positions write to the states or read from them: (B, T, G, N) tokens, (B, G, N, T) or (B, G, N, H, W) planes.
struct StateMap {
    wtconv_ssm_tensor t;
    int64_t G, N;
};
StateMap state_map(const Tensor &t, const char *name, const Dims &d, const Tensor &x) {
    const bool planes = d.layout == WTCONV_SCAN_PLANES;
    const std::string what(name);
    if (t.device() != x.device() || t.scalar_type() != x.scalar_type()) refuse(what + " must match x's dtype and device");
    if (t.dim() != 4 && !(planes && t.dim() == 5)) refuse(what + " must be (B, T, G, N) tokens, or (B, G, N, T) or (B, G, N, H, W) planes");
    const int64_t positions = planes ? (t.dim() == 5 ? t.size(3) * t.size(4) : t.size(3)) : t.size(1);
    const int g = planes ? 1 : 2, n = g + 1;
    if (t.size(0) != d.B || positions != d.T || t.numel() == 0) refuse(what + " must have x's batch and positions");
    const int64_t G = t.size(g), N = t.size(n);
    if (G > INT_MAX || N > INT_MAX) refuse(what + " is too large");
    int64_t row;
    if (planes) {
        if (t.dim() == 5 && ((t.stride(4) != 1 && t.size(4) > 1) || (t.stride(3) != t.size(4) && t.size(3) > 1)))
            refuse(what + ": the pixels of a plane must be contiguous");
        if (t.dim() == 4 && t.stride(3) != 1 && t.size(3) > 1) refuse(what + ": the innermost axis must be contiguous");
        row = N > 1 ? t.stride(2) : t.stride(1);
        if (G > 1 && N > 1 && t.stride(1) != N * row) refuse(what + ": groups must follow one another");
    } else {
        row = t.stride(1);
        if ((N > 1 && t.stride(3) != 1) || (G > 1 && t.stride(2) != N)) refuse(what + ": groups and states must be contiguous");
    }
    return {{t.data_ptr(), (long long)t.stride(0), (long long)row}, G, N};
}

struct Selective {
    wtconv_selective_shape shape;
    wtconv_selective_inputs in;
};
Selective selective(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm, const Given &D, const Given &z,
                    const Given &dt_bias, const Given &lengths, bool softplus, bool planes) {
    Selective s = {};
    s.in.x = ssm(activation(x, "x", planes));
    const Dims d = dims_of(x, planes);
    const c10::Device dev = x.device();
    const StateMap b = state_map(Bm, "B", d, x), c = state_map(Cm, "C", d, x);
    if (b.G != c.G || b.N != c.N) refuse("B and C must have the same groups and states");
    if (d.C % b.G != 0) refuse("x's channels must be a multiple of B's groups");
    s.shape = {d.B, d.T, d.C, (int)b.N, (int)b.G, d.layout, d.dtype, softplus ? 1 : 0};
    s.in.dt = ssm(activation(dt, "dt", planes, &x)), s.in.Bm = b.t, s.in.Cm = c.t;
    s.in.z = ssm_activation(z, "z", planes, x);
    s.in.A = array<float>(A, "A", {d.C, b.N}, dev), s.in.D = array<float>(D, "D", {d.C}, dev);
    s.in.dt_bias = array<float>(dt_bias, "dt_bias", {d.C}, dev), s.in.lengths = array<int>(lengths, "lengths", {d.B}, dev);
    return s;
}

// (of a shape that the library refuses: none, and the call then says why)
std::vector<int64_t> selective_states_shape(const wtconv_selective_shape &s) {
    const int64_t keep = (s.T + WTCONV_SELECTIVE_KEEP - 1) / WTCONV_SELECTIVE_KEEP;
    return {s.B, keep, s.C, (int64_t)(wtconv_selective_states_size(&s) / ((size_t)s.B * keep * s.C))};
}

py::tuple selective_forward(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm, const Given &D,
                            const Given &z, const Given &dt_bias, const Given &h0, const Given &lengths, const std::string &layout,
                            bool softplus, bool keep_states, const Given &y_given, const Given &workspace, const py::object &stream) {
    const bool planes = is_planes(layout);
    Selective s = selective(x, dt, A, Bm, Cm, D, z, dt_bias, lengths, softplus, planes);
    const c10::Device dev = x.device();
    s.in.h0 = array<float>(h0, "h0", {s.shape.B, s.shape.C, s.shape.N}, dev);
    const Call call(stream, dev);
    const Tensor y = y_given.has_value() ? *y_given : call.empty(x.sizes(), x.scalar_type());
    const wtconv_ssm_tensor ay = ssm(activation(y, "y", planes, &x));
    const Tensor h_last = call.empty({s.shape.B, s.shape.C, s.shape.N}, at::kFloat);
    Tensor states;
    if (keep_states) states = call.empty(selective_states_shape(s.shape), at::kFloat);
    const Scratch ws = scratch(workspace, wtconv_selective_workspace_size(WTCONV_SCAN_OP_FORWARD, &s.shape), dev, call);
    call.uses(x, dt, A, Bm, Cm, D, z, dt_bias, h0, lengths, y_given);
    check_status(wtconv_selective_forward(&s.shape, &s.in, &ay, h_last.data_ptr<float>(), keep_states ? states.data_ptr<float>() : nullptr,
                                          ws.p, ws.bytes, call.stream()),
                 "wtconv_selective_forward");
    written(y_given);
    return py::make_tuple(y, h_last, keep_states ? py::cast(states) : py::none());
}

py::tuple selective_backward(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm, const Given &states,
                             const Tensor &dy, const Given &D, const Given &z, const Given &dt_bias, const Given &dh_last,
                             const Given &lengths, const std::string &layout, bool softplus, const Given &dx_given,
                             const Given &d_dt_given, const Given &dB_given, const Given &dC_given, const Given &dz_given,
                             const Given &workspace, const py::object &stream) {
    const bool planes = is_planes(layout);
    const Selective s = selective(x, dt, A, Bm, Cm, D, z, dt_bias, lengths, softplus, planes);
    const c10::Device dev = x.device();
    const int64_t B = s.shape.B, C = s.shape.C, N = s.shape.N;
    if (!states.has_value()) refuse("the backward needs the states of a forward with keep_states=True");
    const float *states_p = array<float>(states, "states", selective_states_shape(s.shape), dev);
    const float *dh_p = array<float>(dh_last, "dh_last", {B, C, N}, dev);
    const wtconv_ssm_tensor ady = ssm(activation(dy, "dy", planes, &x));
    if (dz_given.has_value() && !z.has_value()) refuse("dz is the gradient of z, which is not given");
    const Call call(stream, dev);
    const auto like = [&](const Given &given, const Tensor &t) { return given.has_value() ? *given : call.empty(t.sizes(), t.scalar_type()); };
    const Tensor dx = like(dx_given, x), d_dt = like(d_dt_given, x), dB = like(dB_given, Bm), dC = like(dC_given, Cm);
    const Tensor dA = call.empty({C, N}, at::kFloat), dh0 = call.empty({B, C, N}, at::kFloat);
    Tensor dz, dD, d_bias;
    if (z.has_value()) dz = like(dz_given, x);
    if (D.has_value()) dD = call.empty({C}, at::kFloat);
    if (dt_bias.has_value()) d_bias = call.empty({C}, at::kFloat);
    const Dims d = dims_of(x, planes);
    wtconv_selective_grads g = {};
    g.dx = ssm(activation(dx, "dx", planes, &x)), g.d_dt = ssm(activation(d_dt, "d_dt", planes, &x));
    const StateMap mb = state_map(dB, "dB", d, x), mc = state_map(dC, "dC", d, x);
    if (mb.G != s.shape.G || mb.N != N || mc.G != s.shape.G || mc.N != N) refuse("dB and dC must have the shape of B and C");
    g.dB = mb.t, g.dC = mc.t;
    if (dz.defined()) g.dz = ssm(activation(dz, "dz", planes, &x));
    g.dA = dA.data_ptr<float>(), g.d_h0 = dh0.data_ptr<float>();
    if (dD.defined()) g.dD = dD.data_ptr<float>();
    if (d_bias.defined()) g.d_dt_bias = d_bias.data_ptr<float>();
    const Scratch ws = scratch(workspace, wtconv_selective_workspace_size(WTCONV_SCAN_OP_BACKWARD, &s.shape), dev, call);
    call.uses(x, dt, A, Bm, Cm, states, dy, D, z, dt_bias, dh_last, lengths, dx_given, d_dt_given, dB_given, dC_given, dz_given);
    check_status(wtconv_selective_backward(&s.shape, &s.in, states_p, &ady, dh_p, &g, ws.p, ws.bytes, call.stream()),
                 "wtconv_selective_backward");
    for (const Given *t : {&dx_given, &d_dt_given, &dB_given, &dC_given, &dz_given}) written(*t);
    const auto or_none = [](const Tensor &t) { return t.defined() ? py::cast(t) : py::none(); };
    return py::make_tuple(dx, d_dt, dA, dB, dC, or_none(dD), or_none(dz), or_none(d_bias), dh0);
}

// One position's activations: (B, C), contiguous along C.
void check_rows(const Tensor &x) {
    if (x.dim() != 2 || x.numel() == 0 || !x.is_cuda() || dtype_code(x.scalar_type()) < 0 || x.size(0) > INT_MAX || x.size(1) > INT_MAX)
        refuse("x must be a non-empty (B, C) CUDA tensor of fp32, bf16 or fp16");
}
wtconv_ssm_tensor row_of(const Tensor &t, const char *name, const Tensor &x) {
    if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.device() != x.device() || (t.stride(1) != 1 && x.size(1) > 1))
        refuse(std::string(name) + " must match x's shape, dtype and device and be contiguous along C");
    return {t.data_ptr(), 0, (long long)t.stride(0)};
}

Tensor selective_step(const Tensor &x, const Tensor &dt, const Tensor &A, const Tensor &Bm, const Tensor &Cm, const Tensor &pool,
                      const Given &D, const Given &z, const Given &dt_bias, const Given &slots, bool softplus, const Given &y_given,
                      const py::object &stream) {
    check_rows(x);
    const int64_t B = x.size(0), C = x.size(1);
    const c10::Device dev = x.device();
    const Call call(stream, dev);
    const Tensor y = y_given.has_value() ? *y_given : call.empty({B, C}, x.scalar_type());
    const auto map = [&](const Tensor &t, const char *name) -> wtconv_ssm_tensor {
        if (t.dim() != 3 || t.size(0) != B || t.numel() == 0 || t.scalar_type() != x.scalar_type() || t.device() != dev ||
            t.size(1) > INT_MAX || t.size(2) > INT_MAX)
            refuse(std::string(name) + " must be (B, G, N) of x's dtype and device");
        if ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
            refuse(std::string(name) + ": groups and states must be contiguous");
        return {t.data_ptr(), 0, (long long)t.stride(0)};
    };
    wtconv_selective_inputs in = {};
    in.x = row_of(x, "x", x), in.dt = row_of(dt, "dt", x), in.Bm = map(Bm, "B"), in.Cm = map(Cm, "C");
    const int64_t G = Bm.size(1), N = Bm.size(2);
    if (Cm.size(1) != G || Cm.size(2) != N) refuse("B and C must have the same groups and states");
    if (C % G != 0) refuse("x's channels must be a multiple of B's groups");
    if (z.has_value()) in.z = row_of(*z, "z", x);
    const wtconv_ssm_tensor ay = row_of(y, "y", x);
    if (pool.dim() != 3 || pool.size(1) != C || pool.size(2) != N || pool.size(0) < 1 || pool.size(0) > INT_MAX)
        refuse("pool must be (n_states, " + std::to_string(C) + ", " + std::to_string(N) + ")");
    in.A = array<float>(A, "A", {C, N}, dev), in.D = array<float>(D, "D", {C}, dev), in.dt_bias = array<float>(dt_bias, "dt_bias", {C}, dev);
    float *pool_p = array<float>(pool, "pool", pool.sizes(), dev);
    const int *slots_p = array<int>(slots, "slots", {B}, dev);
    const wtconv_selective_shape shape = {(int)B, 1, (int)C, (int)N, (int)G, WTCONV_SCAN_TOKENS, dtype_code(x.scalar_type()), softplus ? 1 : 0};
    call.uses(x, dt, A, Bm, Cm, pool, D, z, dt_bias, slots, y_given);
    check_status(wtconv_selective_step(&shape, &in, pool_p, (int)pool.size(0), slots_p, &ay, call.stream()), "wtconv_selective_step");
    written(pool), written(y_given);
    return y;
}

// --------------------------------------------------------------------------------- causal convolution

struct Causal {
    wtconv_causal_shape shape;
    wtconv_ssm_tensor x;
    const float *w, *bias;
    const void *state;
    const int *lengths;
    std::vector<int64_t> state_shape;
};
Causal causal(const Tensor &x, const Tensor &weight, const Given &bias, const Given &state, const Given &lengths, bool silu, bool planes) {
    Causal s = {};
    s.x = ssm(activation(x, "x", planes));
    const Dims d = dims_of(x, planes);
    const c10::Device dev = x.device();
    if (weight.dim() != 2 || weight.size(0) != d.C || weight.size(1) < 2 || weight.size(1) > 4)
        refuse("weight must be (" + std::to_string(d.C) + ", K) with K from 2 to 4");
    const int64_t K = weight.size(1);
    s.shape = {d.B, d.T, d.C, (int)K, d.layout, d.dtype, silu ? 1 : 0};
    s.state_shape = {d.B, d.C, K - 1};
    s.w = array<float>(weight, "weight", {d.C, K}, dev), s.bias = array<float>(bias, "bias", {d.C}, dev);
    s.state = like_array(state, "state", s.state_shape, x), s.lengths = array<int>(lengths, "lengths", {d.B}, dev);
    return s;
}

py::tuple causal_forward(const Tensor &x, const Tensor &weight, const Given &bias, const Given &state, const Given &lengths,
                         const std::string &layout, bool silu, const Given &y_given, const py::object &stream) {
    const bool planes = is_planes(layout);
    const Causal s = causal(x, weight, bias, state, lengths, silu, planes);
    const Call call(stream, x.device());
    const Tensor y = y_given.has_value() ? *y_given : call.empty(x.sizes(), x.scalar_type());
    const wtconv_ssm_tensor ay = ssm(activation(y, "y", planes, &x));
    const Tensor last = call.empty(s.state_shape, x.scalar_type());
    call.uses(x, weight, bias, state, lengths, y_given);
    check_status(wtconv_causal_forward(&s.shape, &s.x, s.w, s.bias, s.state, s.lengths, &ay, last.data_ptr(), call.stream()),
                 "wtconv_causal_forward");
    written(y_given);
    return py::make_tuple(y, last);
}

py::tuple causal_backward(const Tensor &x, const Tensor &weight, const Tensor &dy, const Given &bias, const Given &state,
                          const Given &d_last, const Given &lengths, const std::string &layout, bool silu, const Given &dx_given,
                          const Given &workspace, const py::object &stream) {
    const bool planes = is_planes(layout);
    const Causal s = causal(x, weight, bias, state, lengths, silu, planes);
    const c10::Device dev = x.device();
    const wtconv_ssm_tensor ady = ssm(activation(dy, "dy", planes, &x));
    const void *d_last_p = like_array(d_last, "d_last", s.state_shape, x);
    const Call call(stream, dev);
    const Tensor dx = dx_given.has_value() ? *dx_given : call.empty(x.sizes(), x.scalar_type());
    const wtconv_ssm_tensor adx = ssm(activation(dx, "dx", planes, &x));
    const Tensor dw = call.empty(weight.sizes(), at::kFloat);
    Tensor db, d_state;
    if (bias.has_value()) db = call.empty({s.shape.C}, at::kFloat);
    if (state.has_value()) d_state = call.empty(s.state_shape, x.scalar_type());
    const Scratch ws = scratch(workspace, wtconv_causal_workspace_size(&s.shape), dev, call);
    call.uses(x, weight, dy, bias, state, d_last, lengths, dx_given);
    check_status(wtconv_causal_backward(&s.shape, &s.x, s.w, s.bias, s.state, s.lengths, &ady, d_last_p, &adx, dw.data_ptr<float>(),
                                        db.defined() ? db.data_ptr<float>() : nullptr, d_state.defined() ? d_state.data_ptr() : nullptr,
                                        ws.p, ws.bytes, call.stream()),
                 "wtconv_causal_backward");
    written(dx_given);
    return py::make_tuple(dx, dw, db.defined() ? py::cast(db) : py::none(), d_state.defined() ? py::cast(d_state) : py::none());
}

Tensor causal_step(const Tensor &x, const Tensor &weight, const Tensor &pool, const Given &bias, const Given &slots, bool silu,
                   const Given &y_given, const py::object &stream) {
    check_rows(x);
    const int64_t B = x.size(0), C = x.size(1);
    const c10::Device dev = x.device();
    if (weight.dim() != 2 || weight.size(0) != C || weight.size(1) < 2 || weight.size(1) > 4)
        refuse("weight must be (" + std::to_string(C) + ", K) with K from 2 to 4");
    const int64_t K = weight.size(1);
    const Call call(stream, dev);
    const Tensor y = y_given.has_value() ? *y_given : call.empty({B, C}, x.scalar_type());
    const wtconv_ssm_tensor ax = row_of(x, "x", x), ay = row_of(y, "y", x);
    const float *w = array<float>(weight, "weight", {C, K}, dev), *bias_p = array<float>(bias, "bias", {C}, dev);
    if (pool.dim() != 3 || pool.size(0) < 1 || pool.size(0) > INT_MAX)
        refuse("pool must be (n_states, " + std::to_string(C) + ", " + std::to_string(K - 1) + ")");
    void *pool_p = like_array(pool, "pool", {pool.size(0), C, K - 1}, x);
    const int *slots_p = array<int>(slots, "slots", {B}, dev);
    const wtconv_causal_shape shape = {(int)B, 1, (int)C, (int)K, WTCONV_SCAN_TOKENS, dtype_code(x.scalar_type()), silu ? 1 : 0};
    call.uses(x, weight, pool, bias, slots, y_given);
    check_status(wtconv_causal_step(&shape, &ax, w, bias_p, pool_p, (int)pool.size(0), slots_p, &ay, call.stream()), "wtconv_causal_step");
    written(pool), written(y_given);
    return y;
}

// ----------------------------------------------------------------------------------------------- norm

// (..., C) as rows with one stride between them.
wtconv_rms_tensor rows_of(const Tensor &t, const char *name, int64_t &rows) {
    const std::string what(name);
    if (!t.is_cuda() || dtype_code(t.scalar_type()) < 0) refuse(what + " must be a CUDA tensor of fp32, bf16 or fp16");
    if (t.dim() < 1 || t.numel() == 0) refuse(what + " must be (..., C) and not empty");
    const int64_t C = t.size(-1);
    if (C > 1 && t.stride(-1) != 1) refuse(what + ": the innermost axis must be contiguous");
    rows = 1;
    int64_t row = C;
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (rows == 1) row = t.stride(i);
        else if (t.stride(i) != row * rows) refuse(what + ": its rows must lie at one distance from one another");
        rows *= t.size(i);
    }
    if (rows > INT_MAX || C > INT_MAX) refuse(what + " is too large");
    return {t.data_ptr(), (long long)row};
}
wtconv_rms_tensor rows_like(const Tensor &t, const char *name, const Tensor &x, at::ScalarType type) {
    if (t.sizes() != x.sizes() || t.scalar_type() != type || t.device() != x.device())
        refuse(std::string(name) + " must have x's shape and device and be " + c10::toString(type));
    int64_t rows;
    return rows_of(t, name, rows);
}

struct Norm {
    wtconv_rms_shape shape;
    wtconv_rms_tensor x, residual;
    const float *w;
};
Norm norm(const Tensor &x, const Tensor &weight, const Given &residual, double eps) {
    Norm s = {};
    int64_t rows;
    s.x = rows_of(x, "x", rows);
    s.shape = {(int)rows, (int)x.size(-1), dtype_code(x.scalar_type()), dtype_code(x.scalar_type()), (float)eps};
    s.w = array<float>(weight, "weight", {x.size(-1)}, x.device());
    if (residual.has_value()) {
        if (residual->scalar_type() != x.scalar_type() && residual->scalar_type() != at::kFloat)
            refuse("residual must be of x's dtype or fp32");
        s.residual = rows_like(*residual, "residual", x, residual->scalar_type());
        s.shape.total_dtype = dtype_code(residual->scalar_type());
    }
    return s;
}

py::tuple rms_forward(const Tensor &x, const Tensor &weight, const Given &residual, double eps, const Given &y_given,
                      const Given &total_given, const py::object &stream) {
    const Norm s = norm(x, weight, residual, eps);
    if (total_given.has_value() && !residual.has_value()) refuse("without a residual the total is x");
    const Call call(stream, x.device());
    const Tensor y = y_given.has_value() ? *y_given : call.empty(x.sizes(), x.scalar_type());
    const wtconv_rms_tensor ay = rows_like(y, "y", x, x.scalar_type());
    Tensor total = x;
    wtconv_rms_tensor at = {};
    if (residual.has_value()) {
        total = total_given.has_value() ? *total_given : call.empty(x.sizes(), residual->scalar_type());
        at = rows_like(total, "total", x, residual->scalar_type());
    }
    const Tensor rstd = call.empty(x.sizes().slice(0, x.dim() - 1), at::kFloat);
    call.uses(x, weight, residual, y_given, total_given);
    check_status(wtconv_rms_forward(&s.shape, &s.x, &s.residual, s.w, &ay, &at, rstd.data_ptr<float>(), call.stream()), "wtconv_rms_forward");
    written(y_given), written(total_given);
    return py::make_tuple(y, total, rstd);
}

py::tuple rms_forward_e4m3(const Tensor &x, const Tensor &weight, const Given &residual, double eps, int64_t block,
                           const Given &total_given, const py::object &stream) {
    const Norm s = norm(x, weight, residual, eps);
    if (total_given.has_value() && !residual.has_value()) refuse("without a residual the total is x");
    if (block != 0 && block != 128) refuse("block must be 0 (one scale a row) or 128");
    const Call call(stream, x.device());
    const Tensor q = call.empty(x.sizes(), at::kFloat8_e4m3fn);
    std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = block ? (x.size(-1) + block - 1) / block : 1;
    const Tensor scales = call.empty(shape, at::kFloat);
    Tensor total;
    wtconv_rms_tensor at = {};
    if (residual.has_value()) {
        total = total_given.has_value() ? *total_given : call.empty(x.sizes(), residual->scalar_type());
        at = rows_like(total, "total", x, residual->scalar_type());
    }
    call.uses(x, weight, residual, total_given);
    check_status(wtconv_rms_forward_e4m3(&s.shape, &s.x, &s.residual, s.w, (int)block, q.data_ptr(), scales.data_ptr<float>(), &at, call.stream()),
                 "wtconv_rms_forward_e4m3");
    written(total_given);
    return py::make_tuple(q, scales, total.defined() ? py::cast(total) : py::none());
}

py::tuple rms_backward(const Tensor &dy, const Tensor &total, const Tensor &weight, const Tensor &rstd, const Given &d_total, bool residual,
                       const Given &workspace, const py::object &stream) {
    const c10::Device dev = dy.device();
    int64_t rows;
    const wtconv_rms_tensor ady = rows_of(dy, "dy", rows);
    if (total.scalar_type() != dy.scalar_type() && total.scalar_type() != at::kFloat) refuse("total must be of dy's dtype or fp32");
    const wtconv_rms_tensor at = rows_like(total, "total", dy, total.scalar_type());
    wtconv_rms_tensor adt = {}, adx = {}, adr = {};
    if (d_total.has_value()) adt = rows_like(*d_total, "d_total", dy, total.scalar_type());
    const float *w = array<float>(weight, "weight", {dy.size(-1)}, dev);
    const float *rstd_p = array<float>(rstd, "rstd", dy.sizes().slice(0, dy.dim() - 1), dev);
    const wtconv_rms_shape shape = {(int)rows, (int)dy.size(-1), dtype_code(dy.scalar_type()), dtype_code(total.scalar_type()), 0.f};
    const Call call(stream, dev);
    // (of one type, the gradients of x and of the residual are one tensor)
    const Tensor dx = call.empty(dy.sizes(), dy.scalar_type());
    adx = rows_like(dx, "dx", dy, dy.scalar_type());
    Tensor d_residual = dx;
    if (total.scalar_type() != dy.scalar_type()) {
        d_residual = call.empty(dy.sizes(), total.scalar_type());
        adr = rows_like(d_residual, "d_residual", dy, total.scalar_type());
    }
    const Tensor dw = call.empty({dy.size(-1)}, at::kFloat);
    const Scratch ws = scratch(workspace, wtconv_rms_workspace_size(&shape), dev, call);
    call.uses(dy, total, weight, rstd, d_total);
    check_status(wtconv_rms_backward(&shape, &ady, &at, w, rstd_p, &adt, &adx, &adr, dw.data_ptr<float>(), ws.p, ws.bytes, call.stream()),
                 "wtconv_rms_backward");
    return py::make_tuple(dx, residual ? py::cast(d_residual) : py::none(), dw);
}

}  // namespace

void define_mixers(py::module_ &m) {
    m.def("selective_forward", &selective_forward);
    m.def("selective_backward", &selective_backward);
    m.def("selective_step", &selective_step);
    m.def("causal_forward", &causal_forward);
    m.def("causal_backward", &causal_backward);
    m.def("causal_step", &causal_step);
    m.def("rms_forward", &rms_forward);
    m.def("rms_forward_e4m3", &rms_forward_e4m3);
    m.def("rms_backward", &rms_backward);
}
