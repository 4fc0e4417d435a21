// Arguments and launch functions of the root-mean-square norm (wtconv_norm.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "train_common.h"
#include "wtconv_norm.h"

namespace wtconv {

struct NormArgs {
    wtconv_rms_shape s;
    wtconv_rms_tensor x, residual, y, total;           // forward
    wtconv_rms_tensor dy, d_total, dx, d_residual;     // backward (total: an input)
    const float *w, *rstd_in;
    float *rstd, *scales, *dw;
    unsigned char *q;    // e4m3 instead of y
    int block, blocks;   // elements that share a scale (0: a row), scales of a row
    bool wide;           // rows start at multiples of 16 bytes
    float *part;         // [grid][C]: dw of a CTA's rows
};

// CTAs of the backward for this shape, 1024 threads to an SM, or fewer where there are fewer rows.  As many run at once with 512
// < C <= 2048; with other widths registers let a half to three quarters of them, and the others follow.
int norm_backward_grid(int rows, int C);

// T: of the activations, R: of the residual stream
template <typename T, typename R> cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t st);
template <typename T, typename R> cudaError_t launch_norm_backward(const NormArgs &a, cudaStream_t st);

}  // namespace wtconv
