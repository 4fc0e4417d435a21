// Tensor tables and launch functions of the AdamW step and the gradient norm.
#pragma once

#include <cuda_runtime.h>

#include "train_common.h"
#include "wtconv_optim.h"

namespace wtconv {

constexpr int kChunk = 2048;  // elements of one work item: eight warps, one 8-bit block each

// The tensors of one launch, passed as a kernel parameter (constant memory: no upload, and a
// captured graph keeps its own copy).  first[i] is tensor i's first chunk; first[count] the total.
template <int CAP> struct TensorTable {
    wtconv_optim_tensor t[CAP];
    int first[CAP + 1];
    int count;
};
// Two capacities, because a launch copies all of its parameters: 56 tensors and the step's scalars stay
// within 4 KB, 448 are the most that fit the 32,764 bytes of a kernel's parameters.  A step over 25, 40 and
// 56 tensors of 1000 elements, called in a row, takes 3.6, 4.1 and 4.5 us with the small table and 4.5, 5.0
// and 5.4 with the large one (in a graph 2.80, 2.83, 2.92 and 2.83, 2.96, 3.02).  A table of 96 gains another
// 0.6 us from 57 tensors on and costs 0.1 below; one of 24 costs as much as 56 in calls, in a graph 0.2 less.
constexpr int kSmallTable = 56, kLargeTable = 448;

static_assert(sizeof(TensorTable<kLargeTable>) <= 32764 - 128, "the table and the scalars fit a kernel's parameters");

struct StepScalars {
    float beta1, one_minus_beta1, beta2, one_minus_beta2;
    float keep;       // 1 - lr weight_decay
    float rate;       // lr / (1 - beta1^t)
    float root_scale; // 1 / sqrt(1 - beta2^t)
    float eps;
    float negative_zero;  // for `product` (train_device.cuh)
    uint32_t threshold0;  // t K2, the step's part of the rounding threshold
    int state_bits, grad_dtype, copy_dtype;
};
static_assert(sizeof(TensorTable<kSmallTable>) + sizeof(StepScalars) + sizeof(void *) <= 4096, "");

// Part of the norm: chunks of one table summed into `blocks` doubles at part.
int norm_blocks(long long chunks);

template <int CAP> cudaError_t launch_adamw(const TensorTable<CAP> &table, const StepScalars &s, const float *clip, cudaStream_t st);
template <int CAP>
cudaError_t launch_norm_part(const TensorTable<CAP> &table, int grad_dtype, double *part, int blocks, cudaStream_t st);
// The whole norm in one launch, for one table of at most kSmallNorm chunks: 255 fp32 tensors of 1500
// elements 7.5 us with one launch, 300 of them 8.0 with two; one tensor of 522,240 elements 5.5 us with
// one, of 524,289 6.7 with two.
constexpr int kSmallNorm = 256;
template <int CAP>
cudaError_t launch_norm_small(const TensorTable<CAP> &table, int grad_dtype, double max_norm, float *out, cudaStream_t st);
cudaError_t launch_norm_final(const double *part, int count, double max_norm, float *out, cudaStream_t st);
// param / copy of each descriptor stand for m_out / v_out
template <int CAP> cudaError_t launch_state_values(const TensorTable<CAP> &table, cudaStream_t st);

}  // namespace wtconv
