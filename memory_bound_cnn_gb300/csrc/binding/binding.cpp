// Python binding of the operators beside the WTConv layer (include/wtconv_scan.h, wtconv_optim.h; those of
// wtconv_ssm.h and wtconv_norm.h are in mixers.cpp): checks tensors, allocates outputs and scratch from PyTorch's
// caching allocator, and calls the C ABI on the current stream.  Compiled, because these calls are short: a decoding
// step takes 4.5 us of host time here and took 23 us through ctypes.
#include <algorithm>
#include <cstddef>
#include <vector>

#include "common.h"
#include "wtconv_optim.h"

using namespace binding;

void define_mixers(py::module_ &m);  // mixers.cpp

namespace {

// ------------------------------------------------------------------------------------------- scan

std::vector<int64_t> states_shape(const Dims &d) {
    const int64_t n = (d.T + WTCONV_SCAN_KEEP - 1) / WTCONV_SCAN_KEEP;
    if (d.layout == WTCONV_SCAN_PLANES) return {d.B, d.C, n};
    return {d.B, n, d.C};
}

py::tuple scan_forward(const Tensor &x, const Tensor &gate, const Tensor &gate_bias, const optional<Tensor> &h0,
                       const optional<Tensor> &lengths, const std::string &layout, bool keep_states,
                       const optional<Tensor> &y_given, const optional<Tensor> &workspace, const py::object &stream) {
    const bool planes = is_planes(layout);
    const Act ax = activation(x, "x", planes), ag = activation(gate, "gate", planes, &x);
    const Dims d = dims_of(x, planes);
    const c10::Device dev = x.device();
    const float *bias_p = array<float>(gate_bias, "gate_bias", {d.C}, dev);
    const float *h0_p = array<float>(h0, "h0", {d.B, d.C}, dev);
    const int *len_p = array<int>(lengths, "lengths", {d.B}, dev);
    const Call call(stream, dev);
    const Tensor y = y_given.has_value() ? *y_given : call.empty(x.sizes(), x.scalar_type());
    const Act ay = activation(y, "y", planes, &x);
    const Tensor h_last = call.empty({d.B, d.C}, at::kFloat);
    Tensor states;
    if (keep_states) states = call.empty(states_shape(d), at::kFloat);
    const Scratch ws = scratch(workspace, wtconv_scan_workspace_size(WTCONV_SCAN_OP_FORWARD, d.B, d.T, d.C, d.layout, d.dtype), dev, call);
    call.uses(x, gate, gate_bias, h0, lengths, y_given);
    check_status(wtconv_scan_forward(d.B, d.T, d.C, d.layout, d.dtype, ax.p, ax.batch, ax.row, ag.p, ag.batch, ag.row, bias_p,
                                     h0_p, len_p, ay.p, ay.batch, ay.row, h_last.data_ptr<float>(),
                                     keep_states ? states.data_ptr<float>() : nullptr, ws.p, ws.bytes, call.stream()),
                 "wtconv_scan_forward");
    written(y_given);
    return py::make_tuple(y, h_last, keep_states ? py::cast(states) : py::none());
}

py::tuple scan_backward(const Tensor &x, const Tensor &gate, const Tensor &gate_bias, const optional<Tensor> &states,
                        const Tensor &dy, const optional<Tensor> &dh_last, const optional<Tensor> &lengths,
                        const std::string &layout, const optional<Tensor> &dx_given, const optional<Tensor> &d_gate_given,
                        const optional<Tensor> &workspace, const py::object &stream) {
    const bool planes = is_planes(layout);
    const Act ax = activation(x, "x", planes), ag = activation(gate, "gate", planes, &x), ady = activation(dy, "dy", planes, &x);
    const Dims d = dims_of(x, planes);
    const c10::Device dev = x.device();
    if (!states.has_value()) refuse("the backward needs the states of a forward with keep_states=True");
    const float *bias_p = array<float>(gate_bias, "gate_bias", {d.C}, dev);
    const float *states_p = array<float>(states, "states", states_shape(d), dev);
    const float *dh_p = array<float>(dh_last, "dh_last", {d.B, d.C}, dev);
    const int *len_p = array<int>(lengths, "lengths", {d.B}, dev);
    const Call call(stream, dev);
    const Tensor dx = dx_given.has_value() ? *dx_given : call.empty(x.sizes(), x.scalar_type());
    const Tensor d_gate = d_gate_given.has_value() ? *d_gate_given : call.empty(x.sizes(), x.scalar_type());
    const Act adx = activation(dx, "dx", planes, &x), adg = activation(d_gate, "d_gate", planes, &x);
    const Tensor d_bias = call.empty({d.C}, at::kFloat), d_h0 = call.empty({d.B, d.C}, at::kFloat);
    const Scratch ws = scratch(workspace, wtconv_scan_workspace_size(WTCONV_SCAN_OP_BACKWARD, d.B, d.T, d.C, d.layout, d.dtype), dev, call);
    call.uses(x, gate, gate_bias, states, dy, dh_last, lengths, dx_given, d_gate_given);
    check_status(wtconv_scan_backward(d.B, d.T, d.C, d.layout, d.dtype, ax.p, ax.batch, ax.row, ag.p, ag.batch, ag.row, bias_p,
                                      states_p, len_p, ady.p, ady.batch, ady.row, dh_p, adx.p, adx.batch, adx.row, adg.p,
                                      adg.batch, adg.row, d_bias.data_ptr<float>(), d_h0.data_ptr<float>(), ws.p, ws.bytes,
                                      call.stream()),
                 "wtconv_scan_backward");
    written(dx_given), written(d_gate_given);
    return py::make_tuple(dx, d_gate, d_bias, d_h0);
}

Tensor scan_step(const Tensor &x, const Tensor &gate, const Tensor &gate_bias, const Tensor &pool,
                 const optional<Tensor> &slots, const optional<Tensor> &y_given, const py::object &stream) {
    if (x.dim() != 2 || x.numel() == 0 || !x.is_cuda() || dtype_code(x.scalar_type()) < 0 || x.size(0) > INT_MAX ||
        x.size(1) > INT_MAX)
        refuse("x must be a non-empty (B, C) CUDA tensor of fp32, bf16 or fp16");
    const int64_t B = x.size(0), C = x.size(1);
    const c10::Device dev = x.device();
    const Call call(stream, dev);
    const Tensor y = y_given.has_value() ? *y_given : call.empty({B, C}, x.scalar_type());
    const auto check = [&](const Tensor &t, const char *name) {
        if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.device() != dev || (t.stride(1) != 1 && C > 1))
            refuse(std::string(name) + " must match x's shape, dtype and device and be contiguous along C");
    };
    check(x, "x"), check(gate, "gate"), check(y, "y");
    if (pool.dim() != 2 || pool.size(1) != C || pool.size(0) < 1 || pool.size(0) > INT_MAX)
        refuse("pool must be (n_states, " + std::to_string(C) + ")");
    const float *bias_p = array<float>(gate_bias, "gate_bias", {C}, dev);
    float *pool_p = array<float>(pool, "pool", pool.sizes(), dev);
    const int *slots_p = array<int>(slots, "slots", {B}, dev);
    call.uses(x, gate, gate_bias, pool, slots, y_given);
    check_status(wtconv_scan_step((int)B, (int)C, dtype_code(x.scalar_type()), x.data_ptr(), x.stride(0), gate.data_ptr(),
                                  gate.stride(0), bias_p, pool_p, (int)pool.size(0), slots_p, y.data_ptr(), y.stride(0),
                                  call.stream()),
                 "wtconv_scan_step");
    written(pool), written(y_given);
    return y;
}

// ------------------------------------------------------------------------------------------ AdamW

// The tensors behind an optimiser's descriptors, which lie at `address` in its own memory: field by field,
// checked when they are filled in.
class TensorTable {
  public:
    TensorTable(int n, uintptr_t address, const c10::Device &device)
        : list(reinterpret_cast<wtconv_optim_tensor *>(address)), n(n), device(device) {}

    // One tensor per descriptor, whose addresses go to the field at `offset`.  The tensor has one element
    // for every `per` of the parameter's (which `params` sets the number of); None is allowed where
    // `may_be_none` says so.
    void fill(std::vector<optional<Tensor>> given, size_t offset, at::ScalarType dtype, int64_t per, const std::string &name,
              bool params, bool may_be_none) {
        if ((int)given.size() != n) refuse(std::to_string(given.size()) + " tensors in " + name + " for " + std::to_string(n) + " parameters");
        Field f = {std::move(given), offset, dtype, name, may_be_none};
        const std::vector<optional<Tensor>> &ts = f.ts;
        for (int i = 0; i < n; ++i) f.check(i, params && ts[i].has_value() ? ts[i]->numel() : (list[i].n + per - 1) / per, device);
        if (params) refuse_overlaps(ts, name);
        for (int i = 0; i < n; ++i) {  // (only once all of them are right)
            if (!ts[i].has_value()) continue;
            if (params) list[i].n = ts[i]->numel();
            f.address(list[i]) = ts[i]->data_ptr();
        }
        if (params) params_ = std::move(f);
        else if (offset == offsetof(wtconv_optim_tensor, grad)) grads_ = std::move(f);
        else if (offset == offsetof(wtconv_optim_tensor, copy)) copies_ = std::move(f);
    }
    // Before every use: tensors whose memory is another by now (`p.data = ...` gives one a new storage)
    // are checked again and followed.
    void follow_grads() { follow(grads_); }
    void follow() { follow(params_), follow(grads_), follow(copies_); }
    // After a step: the parameters and their copies have changed.
    void stepped() const {
        for (const Field *f : {&params_, &copies_})
            for (const optional<Tensor> &t : f->ts) written(t);
    }

    wtconv_optim_tensor *const list;
    const int n;
    const c10::Device device;

  private:
    struct Field {
        std::vector<optional<Tensor>> ts;
        size_t offset;
        at::ScalarType dtype;
        std::string name;
        bool may_be_none;
        void *&address(wtconv_optim_tensor &t) const { return *reinterpret_cast<void **>(reinterpret_cast<char *>(&t) + offset); }
        void check(int i, int64_t want, const c10::Device &device) const {
            const optional<Tensor> &t = ts[i];
            if (!t.has_value() && may_be_none) return;
            if (!t.has_value() || !t->is_cuda() || t->device() != device || t->scalar_type() != dtype || t->numel() != want ||
                !t->is_contiguous())
                refuse(name + "[" + std::to_string(i) + "] must be a contiguous " + c10::toString(dtype) + " tensor of " +
                       std::to_string(want) + " elements on " + device.str());
        }
    };
    // Elements that two parameters share would be updated by two warps at once.
    static void refuse_overlaps(const std::vector<optional<Tensor>> &ts, const std::string &name) {
        struct Range {
            const char *begin, *end;
            int which;
        };
        std::vector<Range> ranges;
        ranges.reserve(ts.size());
        for (int i = 0; i < (int)ts.size(); ++i) {
            const char *const p = static_cast<const char *>(ts[i]->const_data_ptr());
            if (ts[i]->numel() > 0) ranges.push_back({p, p + ts[i]->nbytes(), i});
        }
        std::sort(ranges.begin(), ranges.end(), [](const Range &a, const Range &b) { return a.begin < b.begin; });
        for (size_t i = 1; i < ranges.size(); ++i)
            if (ranges[i].begin < ranges[i - 1].end)
                refuse(name + "[" + std::to_string(std::min(ranges[i - 1].which, ranges[i].which)) + "] and " + name + "[" +
                       std::to_string(std::max(ranges[i - 1].which, ranges[i].which)) + "] share memory");
    }
    void follow(const Field &f) {
        for (int i = 0; i < (int)f.ts.size(); ++i) {
            const optional<Tensor> &t = f.ts[i];
            if (!t.has_value() || (t->const_data_ptr() == f.address(list[i]) && t->numel() == list[i].n)) continue;
            f.check(i, list[i].n, device);
            f.address(list[i]) = t->data_ptr();
        }
    }
    Field params_, grads_, copies_;
};

Tensor grad_norm(TensorTable &table, int grad_dtype, double max_norm, const optional<Tensor> &out_given,
                 const optional<Tensor> &workspace, size_t workspace_bytes, const py::object &stream) {
    const c10::Device dev = table.device;
    table.follow_grads();
    const Call call(stream, dev);
    const Tensor out = out_given.has_value() ? *out_given : call.empty({2}, at::kFloat);
    float *out_p = array<float>(out, "out", {2}, dev);
    const Scratch ws = scratch(workspace, workspace_bytes, dev, call);
    call.uses(out_given);
    // (scratch: none for few elements)
    check_status(wtconv_grad_norm(table.n, table.list, grad_dtype, max_norm, out_p, ws.p, ws.bytes, call.stream()),
                 "wtconv_grad_norm");
    written(out_given);
    return out;
}

// config: address of the optimiser's wtconv_adamw_config, which takes the step's rate and number.
void adamw_step(TensorTable &table, uintptr_t config_address, double lr, long long step, const optional<Tensor> &clip,
                const py::object &stream) {
    wtconv_adamw_config *const config = reinterpret_cast<wtconv_adamw_config *>(config_address);
    config->lr = lr, config->step = step;
    const c10::Device dev = table.device;
    const float *clip_p = array<float>(clip, "clip", {2}, dev);
    table.follow();
    const Call call(stream, dev);
    call.uses(clip);
    check_status(wtconv_adamw_step(table.n, table.list, config,
                                   clip_p != nullptr ? clip_p + 1 : nullptr, call.stream()),
                 "wtconv_adamw_step");
    table.stepped();
}

// The lists (m, v) where they are new, None for one that the caller gave.
py::tuple state_values(const TensorTable &table, const optional<std::vector<Tensor>> &m_given,
                       const optional<std::vector<Tensor>> &v_given, const py::object &stream) {
    const int n = table.n;
    const c10::Device dev = table.device;
    const Call call(stream, dev);
    std::vector<Tensor> m_new, v_new;
    const auto outputs = [&](const optional<std::vector<Tensor>> &given, std::vector<Tensor> &made) -> const std::vector<Tensor> & {
        if (given.has_value()) return *given;
        for (int i = 0; i < n; ++i) made.push_back(call.empty({(int64_t)table.list[i].n}, at::kFloat));
        return made;
    };
    const auto pointers = [&](const std::vector<Tensor> &ts, const char *name) {
        if ((int)ts.size() != n)
            refuse(std::to_string(ts.size()) + " tensors in " + name + " for " + std::to_string(n) + " parameters");
        std::vector<float *> p(n);
        for (int i = 0; i < n; ++i) {
            const Tensor &t = ts[i];
            if (t.device() != dev || t.scalar_type() != at::kFloat || t.numel() != table.list[i].n || !t.is_contiguous())
                refuse(std::string(name) + "[" + std::to_string(i) + "] must be a contiguous fp32 tensor of " +
                       std::to_string(table.list[i].n) + " elements on " + dev.str());
            call.uses(t);
            p[i] = static_cast<float *>(t.data_ptr());
        }
        return p;
    };
    const std::vector<float *> m = pointers(outputs(m_given, m_new), "m_out"), v = pointers(outputs(v_given, v_new), "v_out");
    check_status(wtconv_adamw_state_values(n, table.list, m.data(), v.data(), call.stream()), "wtconv_adamw_state_values");
    for (const auto *given : {&m_given, &v_given})
        if (given->has_value())
            for (const Tensor &t : **given) written(t);
    return py::make_tuple(m_given.has_value() ? py::none() : py::cast(m_new), v_given.has_value() ? py::none() : py::cast(v_new));
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
    m.def("scan_forward", &scan_forward);
    m.def("scan_backward", &scan_backward);
    m.def("scan_step", &scan_step);
    py::class_<TensorTable>(m, "TensorTable").def(py::init<int, uintptr_t, const c10::Device &>()).def("fill", &TensorTable::fill);
    m.def("grad_norm", &grad_norm);
    m.def("adamw_step", &adamw_step);
    m.def("state_values", &state_values);
    define_mixers(m);
}
