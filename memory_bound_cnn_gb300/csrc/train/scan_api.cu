// C entry points of the gated scan: argument checks, then one of the launch functions.
#include "scan.h"

using namespace wtconv;

namespace {

int check_shape(int B, int T, int C, int layout, int dtype) {
    if (B <= 0 || T <= 0 || C <= 0 || (long long)B * C > 0x7fffffffll || T > (1 << 30)) return WTCONV_ERR_INVALID_ARG;
    if (layout != WTCONV_SCAN_PLANES && layout != WTCONV_SCAN_TOKENS) return WTCONV_ERR_INVALID_ARG;
    return dtype_ok(dtype) ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

bool check_tensor(const ScanTensor &s, const ScanArgs &a, bool output) {
    const long long inner = a.layout == WTCONV_SCAN_PLANES ? a.T : a.C, rows = a.layout == WTCONV_SCAN_PLANES ? a.C : a.T;
    return activation_ok(s.p, s.batch, s.row, a.B, rows, inner, a.dtype, output);
}

ScanTensor input(const void *p, long long batch, long long row) { return {const_cast<void *>(p), batch, row}; }

ScanArgs shape_args(int B, int T, int C, int layout, int dtype) {
    ScanArgs a = {};
    a.B = B, a.T = T, a.C = C, a.layout = layout, a.dtype = dtype;
    a.keep = (T + WTCONV_SCAN_KEEP - 1) / WTCONV_SCAN_KEEP;
    return a;
}

size_t scan_workspace(int op, const ScanArgs &a) {
    return a.layout == WTCONV_SCAN_PLANES ? scan_planes_workspace(op, a) : scan_tokens_workspace(op, a);
}

int check_workspace(int op, const ScanArgs &a, const void *workspace, size_t bytes) {
    const size_t need = scan_workspace(op, a);
    if (need == 0) return WTCONV_OK;
    if (workspace != nullptr && !aligned_to(workspace, 16)) return WTCONV_ERR_INVALID_ARG;
    return workspace == nullptr || bytes < need ? WTCONV_ERR_WORKSPACE : WTCONV_OK;
}

}  // namespace

extern "C" {

size_t wtconv_scan_workspace_size(int op, int B, int T, int C, int layout, int dtype) {
    if (check_shape(B, T, C, layout, dtype) != WTCONV_OK || (op != WTCONV_SCAN_OP_FORWARD && op != WTCONV_SCAN_OP_BACKWARD))
        return 0;
    return scan_workspace(op, shape_args(B, T, C, layout, dtype));
}

int wtconv_scan_status(void) {
    if (cudaDeviceSynchronize() != cudaSuccess) return WTCONV_ERR_CUDA;
    int raised = 0;
    if (take_scan_timeout(&raised) != cudaSuccess) return WTCONV_ERR_CUDA;
    return raised ? WTCONV_ERR_DEVICE_TIMEOUT : WTCONV_OK;
}

int wtconv_scan_selftest_wait_timeout(wtconv_stream_t stream) {
    return status_of(launch_scan_wait_selftest(reinterpret_cast<cudaStream_t>(stream)));
}

int wtconv_scan_forward(int B, int T, int C, int layout, int dtype, const void *x, long long x_batch, long long x_row,
                        const void *gate, long long gate_batch, long long gate_row, const float *gate_bias,
                        const float *h0, const int *lengths, void *y, long long y_batch, long long y_row,
                        float *h_last, float *states, void *workspace, size_t workspace_bytes, wtconv_stream_t stream) {
    int rc = check_shape(B, T, C, layout, dtype);
    if (rc != WTCONV_OK) return rc;
    ScanArgs a = shape_args(B, T, C, layout, dtype);
    a.x = input(x, x_batch, x_row), a.gate = input(gate, gate_batch, gate_row), a.y = {y, y_batch, y_row};
    if (!check_tensor(a.x, a, false) || !check_tensor(a.gate, a, false) || !check_tensor(a.y, a, true) ||
        !f32_ok(gate_bias, false) || !f32_ok(h0, true) || !f32_ok(lengths, true) || !f32_ok(h_last, true) ||
        !f32_ok(states, true))
        return WTCONV_ERR_INVALID_ARG;
    a.gate_bias = gate_bias, a.h0 = h0, a.lengths = lengths, a.h_last = h_last, a.states_out = states;
    a.workspace = workspace;
    if ((rc = check_workspace(WTCONV_SCAN_OP_FORWARD, a, workspace, workspace_bytes)) != WTCONV_OK) return rc;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(layout == WTCONV_SCAN_PLANES ? launch_scan_planes_forward(a, st) : launch_scan_tokens_forward(a, st));
}

int wtconv_scan_backward(int B, int T, int C, int layout, int dtype, const void *x, long long x_batch, long long x_row,
                         const void *gate, long long gate_batch, long long gate_row, const float *gate_bias,
                         const float *states, const int *lengths, const void *dy, long long dy_batch, long long dy_row,
                         const float *dh_last, void *dx, long long dx_batch, long long dx_row, void *d_gate,
                         long long d_gate_batch, long long d_gate_row, float *d_gate_bias, float *d_h0, void *workspace,
                         size_t workspace_bytes, wtconv_stream_t stream) {
    int rc = check_shape(B, T, C, layout, dtype);
    if (rc != WTCONV_OK) return rc;
    ScanArgs a = shape_args(B, T, C, layout, dtype);
    a.x = input(x, x_batch, x_row), a.gate = input(gate, gate_batch, gate_row), a.dy = input(dy, dy_batch, dy_row);
    a.dx = {dx, dx_batch, dx_row}, a.d_gate = {d_gate, d_gate_batch, d_gate_row};
    if (!check_tensor(a.x, a, false) || !check_tensor(a.gate, a, false) || !check_tensor(a.dy, a, false) ||
        !check_tensor(a.dx, a, true) || !check_tensor(a.d_gate, a, true) || !f32_ok(gate_bias, false) ||
        !f32_ok(states, false) || !f32_ok(lengths, true) || !f32_ok(dh_last, true) || !f32_ok(d_gate_bias, false) ||
        !f32_ok(d_h0, true))
        return WTCONV_ERR_INVALID_ARG;
    a.gate_bias = gate_bias, a.states_in = states, a.lengths = lengths, a.dh_last = dh_last;
    a.d_gate_bias = d_gate_bias, a.d_h0 = d_h0, a.workspace = workspace;
    if ((rc = check_workspace(WTCONV_SCAN_OP_BACKWARD, a, workspace, workspace_bytes)) != WTCONV_OK) return rc;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status_of(layout == WTCONV_SCAN_PLANES ? launch_scan_planes_backward(a, st) : launch_scan_tokens_backward(a, st));
}

int wtconv_scan_step(int B, int C, int dtype, const void *x, long long x_row, const void *gate, long long gate_row,
                     const float *gate_bias, float *pool, int n_states, const int *slots, void *y, long long y_row,
                     wtconv_stream_t stream) {
    int rc = check_shape(B, 1, C, WTCONV_SCAN_TOKENS, dtype);
    if (rc != WTCONV_OK) return rc;
    const ScanArgs a = shape_args(B, 1, C, WTCONV_SCAN_TOKENS, dtype);
    const ScanTensor tx = input(x, x_row, 0), tg = input(gate, gate_row, 0), ty = {y, y_row, 0};
    if (!check_tensor(tx, a, false) || !check_tensor(tg, a, false) || !check_tensor(ty, a, true) ||
        !f32_ok(gate_bias, false) || !f32_ok(pool, false) || !f32_ok(slots, true) || n_states <= 0 ||
        (slots == nullptr && n_states < B))
        return WTCONV_ERR_INVALID_ARG;
    if (fault_injected()) return WTCONV_ERR_INJECTED;
    return status_of(launch_scan_step(B, C, dtype, {tx.p, 0, x_row}, {tg.p, 0, gate_row}, gate_bias, pool, n_states, slots,
                                      {y, 0, y_row}, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
