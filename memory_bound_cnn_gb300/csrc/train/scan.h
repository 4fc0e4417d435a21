// Arguments of the gated scan's kernels.
#pragma once

#include <cuda_runtime.h>

#include "train_common.h"
#include "wtconv_scan.h"

namespace wtconv {

// One activation tensor: element strides of its batch and row axes (a row is a channel of planes
// or a position of tokens); the innermost axis is contiguous.
struct ScanTensor {
    void *p;
    long long batch, row;
};

struct ScanArgs {
    int B, T, C, keep;  // keep = kept states per sequence and channel, ceil(T / WTCONV_SCAN_KEEP)
    int layout, dtype;
    ScanTensor x, gate, y;        // forward
    ScanTensor dy, dx, d_gate;    // backward
    const float *gate_bias, *h0, *dh_last, *states_in;
    const int *lengths;
    float *h_last, *states_out, *d_gate_bias, *d_h0;
    void *workspace;
};

// planes (scan_planes.cu) and tokens (scan_tokens.cu)
size_t scan_planes_workspace(int op, const ScanArgs &a);
cudaError_t launch_scan_planes_forward(const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_planes_backward(const ScanArgs &a, cudaStream_t st);
// whether a bounded wait gave up on the current device since the last call; clears it
cudaError_t take_scan_timeout(int *raised);
// a bounded wait that gives up
cudaError_t launch_scan_wait_selftest(cudaStream_t st);
size_t scan_tokens_workspace(int op, const ScanArgs &a);
cudaError_t launch_scan_tokens_forward(const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_tokens_backward(const ScanArgs &a, cudaStream_t st);
cudaError_t launch_scan_step(int B, int C, int dtype, const ScanTensor &x, const ScanTensor &gate, const float *gate_bias,
                             float *pool, int n_states, const int *slots, const ScanTensor &y, cudaStream_t st);

}  // namespace wtconv
