// C entry points of the AdamW step and the gradient norm: argument checks, and the split of the
// tensors into tables that fit a kernel's parameters.
#include <math.h>

#include "optim.h"

using namespace wtconv;

namespace {

constexpr uint32_t kStepStride = 2447445414u;  // 2^32 / p^2, p^3 = p + 1
constexpr long long kMostElements = 1ll << 40;  // of one tensor

long long chunks_of(long long n) { return (n + kChunk - 1) / kChunk; }

// Non-empty tensors from `at` on that one launch takes: at most kLargeTable of them and at most
// 2^30 chunks.
struct Batch {
    int begin, end, count;
    long long chunks;
};
Batch next_batch(int n_tensors, const wtconv_optim_tensor *t, int at) {
    Batch b = {at, at, 0, 0};
    for (; b.end < n_tensors; ++b.end) {
        if (t[b.end].n == 0) continue;
        const long long c = chunks_of(t[b.end].n);
        if (b.count == kLargeTable || b.chunks + c > (1ll << 30)) break;
        ++b.count, b.chunks += c;
    }
    return b;
}

template <int CAP> void fill(TensorTable<CAP> &table, const Batch &b, const wtconv_optim_tensor *t) {
    int k = 0, chunks = 0;
    for (int i = b.begin; i < b.end; ++i) {
        if (t[i].n == 0) continue;
        table.t[k] = t[i];
        table.first[k++] = chunks;
        chunks += (int)chunks_of(t[i].n);
    }
    table.first[k] = chunks;
    table.count = k;
}

// Calls run(table, batch) for table after table, until one fails.
template <typename F> int for_each_table(int n_tensors, const wtconv_optim_tensor *t, F run) {
    for (int at = 0; at < n_tensors;) {
        const Batch b = next_batch(n_tensors, t, at);
        at = b.end;
        if (b.count == 0) continue;
        cudaError_t e;
        if (b.count <= kSmallTable) {
            TensorTable<kSmallTable> table;
            fill(table, b, t);
            e = run(table, b);
        } else {
            TensorTable<kLargeTable> table;
            fill(table, b, t);
            e = run(table, b);
        }
        if (e != cudaSuccess) return WTCONV_ERR_CUDA;
    }
    return WTCONV_OK;
}

bool list_ok(int n_tensors, const wtconv_optim_tensor *t) {
    if (n_tensors <= 0 || t == nullptr) return false;
    for (int i = 0; i < n_tensors; ++i)
        if (t[i].n < 0 || t[i].n > kMostElements) return false;
    return true;
}
// one launch sums every gradient
bool small_norm(int n_tensors, const wtconv_optim_tensor *t) {
    const Batch b = next_batch(n_tensors, t, 0);
    return b.end == n_tensors && b.count > 0 && b.chunks <= kSmallNorm;
}
bool f32_ok(const void *p) { return p != nullptr && aligned_to(p, 4); }
bool state8_ok(const wtconv_optim_tensor &t) {
    return t.m != nullptr && t.v != nullptr && f32_ok(t.m_max) && f32_ok(t.v_max);
}
bool between(double v, double lo, double hi) { return v >= lo && v < hi; }  // false for NaN

}  // namespace

extern "C" {

int wtconv_adamw_step(int n_tensors, const wtconv_optim_tensor *tensors, const wtconv_adamw_config *config,
                      const float *clip, wtconv_stream_t stream) {
    if (!list_ok(n_tensors, tensors) || config == nullptr) return WTCONV_ERR_INVALID_ARG;
    const wtconv_adamw_config &c = *config;
    if (!between(c.lr, 0, INFINITY) || !between(c.eps, 0, INFINITY) || !between(c.weight_decay, 0, INFINITY) ||
        !between(c.beta1, 0, 1) || !between(c.beta2, 0, 1) || c.step < 1 || !aligned_to(clip, 4))
        return WTCONV_ERR_INVALID_ARG;
    if ((c.state_bits != 32 && c.state_bits != 8) || !dtype_ok(c.grad_dtype)) return WTCONV_ERR_UNSUPPORTED;
    for (int i = 0; i < n_tensors; ++i) {
        const wtconv_optim_tensor &t = tensors[i];
        if (t.n == 0) continue;
        if (!f32_ok(t.param) || t.grad == nullptr || !aligned_to(t.grad, elem_bytes_of(c.grad_dtype)) ||
            (c.state_bits == 32 ? !f32_ok(t.m) || !f32_ok(t.v) : !state8_ok(t)))
            return WTCONV_ERR_INVALID_ARG;
        if (t.copy != nullptr && !aligned_to(t.copy, 2)) return WTCONV_ERR_INVALID_ARG;
        if (t.copy != nullptr && c.copy_dtype != WTCONV_BF16 && c.copy_dtype != WTCONV_F16) return WTCONV_ERR_UNSUPPORTED;
    }
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    StepScalars s;
    s.beta1 = (float)c.beta1, s.one_minus_beta1 = (float)(1.0 - c.beta1);
    s.beta2 = (float)c.beta2, s.one_minus_beta2 = (float)(1.0 - c.beta2);
    s.keep = (float)(1.0 - c.lr * c.weight_decay);
    s.rate = (float)(c.lr / (1.0 - pow(c.beta1, (double)c.step)));
    s.root_scale = (float)(1.0 / sqrt(1.0 - pow(c.beta2, (double)c.step)));
    s.eps = (float)c.eps;
    s.negative_zero = -0.f;
    s.threshold0 = (uint32_t)c.step * kStepStride;
    s.state_bits = c.state_bits, s.grad_dtype = c.grad_dtype, s.copy_dtype = c.copy_dtype;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return for_each_table(n_tensors, tensors, [&](const auto &table, const Batch &) { return launch_adamw(table, s, clip, st); });
}

int wtconv_adamw_state_values(int n_tensors, const wtconv_optim_tensor *tensors, float *const *m_out, float *const *v_out,
                              wtconv_stream_t stream) {
    if (!list_ok(n_tensors, tensors) || (m_out == nullptr && v_out == nullptr)) return WTCONV_ERR_INVALID_ARG;
    for (int i = 0; i < n_tensors; ++i)
        if (tensors[i].n > 0 && (!state8_ok(tensors[i]) || (m_out != nullptr && !f32_ok(m_out[i])) ||
                                 (v_out != nullptr && !f32_ok(v_out[i]))))
            return WTCONV_ERR_INVALID_ARG;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return for_each_table(n_tensors, tensors, [&](auto &table, const Batch &b) {
        for (int i = b.begin, k = 0; i < b.end; ++i) {
            if (tensors[i].n == 0) continue;
            table.t[k].param = m_out != nullptr ? m_out[i] : nullptr;
            table.t[k++].copy = v_out != nullptr ? v_out[i] : nullptr;
        }
        return launch_state_values(table, st);
    });
}

size_t wtconv_grad_norm_workspace_size(int n_tensors, const wtconv_optim_tensor *tensors) {
    if (!list_ok(n_tensors, tensors) || small_norm(n_tensors, tensors)) return 0;
    size_t blocks = 0;
    for (int at = 0; at < n_tensors;) {
        const Batch b = next_batch(n_tensors, tensors, at);
        blocks += norm_blocks(b.chunks);
        at = b.end;
    }
    return (blocks * sizeof(double) + 255) / 256 * 256;
}

int wtconv_grad_norm(int n_tensors, const wtconv_optim_tensor *tensors, int grad_dtype, double max_norm, float *out,
                     void *workspace, size_t workspace_bytes, wtconv_stream_t stream) {
    if (!list_ok(n_tensors, tensors) || !f32_ok(out) || !(max_norm > 0)) return WTCONV_ERR_INVALID_ARG;
    if (!dtype_ok(grad_dtype)) return WTCONV_ERR_UNSUPPORTED;
    for (int i = 0; i < n_tensors; ++i)
        if (tensors[i].n > 0 && (tensors[i].grad == nullptr || !aligned_to(tensors[i].grad, elem_bytes_of(grad_dtype))))
            return WTCONV_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned_to(workspace, 16)) return WTCONV_ERR_INVALID_ARG;
    const size_t need = wtconv_grad_norm_workspace_size(n_tensors, tensors);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return WTCONV_ERR_WORKSPACE;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (small_norm(n_tensors, tensors))
        return for_each_table(n_tensors, tensors, [&](const auto &table, const Batch &) {
            return launch_norm_small(table, grad_dtype, max_norm, out, st);
        });
    double *part = static_cast<double *>(workspace);
    int used = 0;
    const int rc = for_each_table(n_tensors, tensors, [&](const auto &table, const Batch &b) {
        const int blocks = norm_blocks(b.chunks);
        const cudaError_t e = launch_norm_part(table, grad_dtype, part + used, blocks, st);
        used += blocks;
        return e;
    });
    if (rc != WTCONV_OK) return rc;
    return status_of(launch_norm_final(part, used, max_norm, out, st));
}

}  // extern "C"
