// Gated scan, one thread per sequence and channel: the recurrence as it is written, position by
// position, for any strides.  Bound by the latency of one position after the other.
#include "scan_device.cuh"

namespace wtconv {

namespace {

constexpr int kRowThreads = 64;

struct Step {  // where element (b, c, t) of a tensor is: base + t * step
    long long base, step;
};
__device__ __forceinline__ Step at(const ScanTensor &s, int layout, int b, int c) {
    return layout == WTCONV_SCAN_PLANES ? Step{b * s.batch + c * s.row, 1} : Step{b * s.batch + c, s.row};
}
__device__ __forceinline__ long long state_at(const ScanArgs &a, int b, int c, int k) {
    return a.layout == WTCONV_SCAN_PLANES ? ((long long)b * a.C + c) * a.keep + k : ((long long)b * a.keep + k) * a.C + c;
}

template <typename T> __global__ void __launch_bounds__(kRowThreads) scan_rows_forward_kernel(ScanArgs a) {
    const long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x;
    if (i >= (long long)a.B * a.C) return;
    const int b = (int)(i / a.C), c = (int)(i - (long long)b * a.C);
    const Step sx = at(a.x, a.layout, b, c), sg = at(a.gate, a.layout, b, c), sy = at(a.y, a.layout, b, c);
    const T *x = static_cast<const T *>(a.x.p) + sx.base, *g = static_cast<const T *>(a.gate.p) + sg.base;
    T *y = static_cast<T *>(a.y.p) + sy.base;
    const float bias = a.gate_bias[c];
    const int n = scan_length(a.lengths, b, a.T);
    float h = a.h0 != nullptr ? a.h0[i] : 0.f;
    for (int t = 0; t < a.T; ++t) {
        if (a.states_out != nullptr && t % WTCONV_SCAN_KEEP == 0) a.states_out[state_at(a, b, c, t / WTCONV_SCAN_KEEP)] = h;
        if (t < n) {
            const Gate q = gate_of(to_f32(g[t * sg.step]) + bias);
            h = fmaf(q.a, h, q.b * to_f32(x[t * sx.step]));
        }
        y[t * sy.step] = from_f32<T>(t < n ? h : 0.f);
    }
    if (a.h_last != nullptr) a.h_last[i] = h;
}

// Two passes over each stretch of WTCONV_SCAN_KEEP positions, last stretch first: h forward from the
// kept state into a local array, then dh backward.
template <typename T> __global__ void __launch_bounds__(kRowThreads) scan_rows_backward_kernel(ScanArgs a) {
    const long long i = (long long)blockIdx.x * kRowThreads + threadIdx.x;
    if (i >= (long long)a.B * a.C) return;
    const int b = (int)(i / a.C), c = (int)(i - (long long)b * a.C);
    const Step sx = at(a.x, a.layout, b, c), sg = at(a.gate, a.layout, b, c), sdy = at(a.dy, a.layout, b, c);
    const Step sdx = at(a.dx, a.layout, b, c), sdg = at(a.d_gate, a.layout, b, c);
    const T *x = static_cast<const T *>(a.x.p) + sx.base, *g = static_cast<const T *>(a.gate.p) + sg.base;
    const T *dy = static_cast<const T *>(a.dy.p) + sdy.base;
    T *dx = static_cast<T *>(a.dx.p) + sdx.base, *dg = static_cast<T *>(a.d_gate.p) + sdg.base;
    const float bias = a.gate_bias[c];
    const int n = scan_length(a.lengths, b, a.T);
    float flow = a.dh_last != nullptr ? a.dh_last[i] : 0.f;  // a_{t+1} dh_{t+1}
    float sum = 0.f;
    float before[WTCONV_SCAN_KEEP];
    for (int k = a.keep - 1; k >= 0; --k) {
        const int t0 = k * WTCONV_SCAN_KEEP, t1 = min(t0 + WTCONV_SCAN_KEEP, a.T);
        float h = a.states_in[state_at(a, b, c, k)];
        for (int t = t0; t < min(t1, n); ++t) {
            const Gate q = gate_of(to_f32(g[t * sg.step]) + bias);
            before[t - t0] = h;
            h = fmaf(q.a, h, q.b * to_f32(x[t * sx.step]));
        }
        for (int t = t1 - 1; t >= t0; --t) {
            float dxv = 0.f, dgv = 0.f;
            if (t < n) {
                const Gate q = gate_of(to_f32(g[t * sg.step]) + bias);
                const float dh = to_f32(dy[t * sdy.step]) + flow;
                dxv = q.b * dh;
                dgv = dh * (before[t - t0] - to_f32(x[t * sx.step])) * (q.a * q.b);
                sum += dgv;
                flow = q.a * dh;
            }
            dx[t * sdx.step] = from_f32<T>(dxv);
            dg[t * sdg.step] = from_f32<T>(dgv);
        }
    }
    if (a.d_h0 != nullptr) a.d_h0[i] = flow;
    static_cast<float *>(a.workspace)[i] = sum;
}

__global__ void __launch_bounds__(256) scan_bias_kernel(const float *part, float *out, int B, int C) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    float s = 0.f;
    for (int b = 0; b < B; ++b) s += part[(long long)b * C + c];
    out[c] = s;
}

template <typename T>
__global__ void __launch_bounds__(256) scan_step_kernel(int C, int parts, ScanTensor x, ScanTensor gate, const float *gate_bias,
                                                        float *pool, int n_states, const int *slots, ScanTensor y) {
    const int b = blockIdx.x / parts, c = (blockIdx.x - b * parts) * 256 + threadIdx.x;
    if (c >= C) return;
    const int slot = slots != nullptr ? slots[b] : b;
    float h = 0.f;
    if (slot >= 0 && slot < n_states) {
        float *s = pool + (long long)slot * C + c;
        const Gate q = gate_of(to_f32(static_cast<const T *>(gate.p)[b * gate.row + c]) + gate_bias[c]);
        h = fmaf(q.a, *s, q.b * to_f32(static_cast<const T *>(x.p)[b * x.row + c]));
        *s = h;
    }
    static_cast<T *>(y.p)[b * y.row + c] = from_f32<T>(h);
}

}  // namespace

size_t scan_tokens_workspace(int op, const ScanArgs &a) {
    return op == WTCONV_SCAN_OP_BACKWARD ? ((size_t)a.B * a.C * sizeof(float) + 255) / 256 * 256 : 0;
}

cudaError_t launch_scan_tokens_forward(const ScanArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)(((long long)a.B * a.C + kRowThreads - 1) / kRowThreads);
    if (a.dtype == WTCONV_F32) scan_rows_forward_kernel<float><<<grid, kRowThreads, 0, st>>>(a);
    else if (a.dtype == WTCONV_BF16) scan_rows_forward_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, st>>>(a);
    else scan_rows_forward_kernel<__half><<<grid, kRowThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_scan_tokens_backward(const ScanArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)(((long long)a.B * a.C + kRowThreads - 1) / kRowThreads);
    if (a.dtype == WTCONV_F32) scan_rows_backward_kernel<float><<<grid, kRowThreads, 0, st>>>(a);
    else if (a.dtype == WTCONV_BF16) scan_rows_backward_kernel<__nv_bfloat16><<<grid, kRowThreads, 0, st>>>(a);
    else scan_rows_backward_kernel<__half><<<grid, kRowThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    scan_bias_kernel<<<(a.C + 255) / 256, 256, 0, st>>>(static_cast<const float *>(a.workspace), a.d_gate_bias, a.B, a.C);
    return cudaGetLastError();
}

cudaError_t launch_scan_step(int B, int C, int dtype, const ScanTensor &x, const ScanTensor &gate, const float *gate_bias,
                             float *pool, int n_states, const int *slots, const ScanTensor &y, cudaStream_t st) {
    const int parts = (C + 255) / 256;
    const unsigned grid = (unsigned)B * parts;
    if (dtype == WTCONV_F32) scan_step_kernel<float><<<grid, 256, 0, st>>>(C, parts, x, gate, gate_bias, pool, n_states, slots, y);
    else if (dtype == WTCONV_BF16)
        scan_step_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(C, parts, x, gate, gate_bias, pool, n_states, slots, y);
    else scan_step_kernel<__half><<<grid, 256, 0, st>>>(C, parts, x, gate, gate_bias, pool, n_states, slots, y);
    return cudaGetLastError();
}

}  // namespace wtconv
