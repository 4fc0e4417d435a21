// Arguments and launch functions of the causal convolution (wtconv_ssm.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "train_common.h"
#include "wtconv_ssm.h"

namespace wtconv {

struct CausalArgs {
    wtconv_causal_shape s;
    wtconv_ssm_tensor x, y, dy, dx;
    const float *w, *bias;
    const void *state, *d_last;  // [B][C][K-1]
    void *state_last, *d_state;
    const int *lengths;
    float *dw, *d_bias;
    bool wide;       // whether addresses and strides allow vectors
    // tokens: a thread takes `strip` positions of a few channels, a CTA 8 strips;
    // planes: 2^row_bits lanes take the vectors of `strip` positions of a row
    int strip, strips, row_bits;
    float *part_w, *part_b;  // [parts][C][K], [parts][C]: a part is a sequence's strips of a CTA, or a row's strip
    int parts;
};

template <typename T> cudaError_t launch_causal_forward(const CausalArgs &a, cudaStream_t st);
template <typename T> cudaError_t launch_causal_backward(const CausalArgs &a, cudaStream_t st);
template <typename T> cudaError_t launch_causal_step(const CausalArgs &a, void *pool, int n_states, const int *slots, cudaStream_t st);

}  // namespace wtconv
