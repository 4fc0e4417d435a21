// Sums of partial results over the parts that different CTAs worked on.
#pragma once

#include "train_common.h"
#include "train_device.cuh"

namespace wtconv {

// out[i] = sum over p < parts of part[p * width + i], in a fixed order: 32 columns to a CTA, 32 threads to a
// column.  A null `out` is left out.
struct ColumnSums {
    const float *part[3];
    float *out[3];
    int width[3], blocks[3];
    int parts;
};
static __global__ void __launch_bounds__(1024) column_sums_kernel(const __grid_constant__ ColumnSums s) {
    __shared__ float meet[32][33];
    begin_kernel();
    int which = 0, block = blockIdx.x;
    while (block >= s.blocks[which]) block -= s.blocks[which++];
    const int width = s.width[which], lane = threadIdx.x % 32, slice = threadIdx.x / 32, i = block * 32 + lane;
    float v = 0.f;
    if (i < width) {
#pragma unroll 8
        for (int p = slice; p < s.parts; p += 32) v += s.part[which][(long long)p * width + i];
    }
    meet[slice][lane] = v;
    __syncthreads();
    v = warp_sum(meet[lane][slice]);
    const int out = block * 32 + slice;
    if (lane == 0 && out < width) s.out[which][out] = v;
}
inline cudaError_t launch_column_sums(ColumnSums s, cudaStream_t st) {
    unsigned blocks = 0;
    for (int i = 0; i < 3; ++i) blocks += s.blocks[i] = s.out[i] == nullptr ? 0 : ceil_div(s.width[i], 32);
    return blocks == 0 ? cudaSuccess : launch_kernel(column_sums_kernel, blocks, 1024, 0, st, 1, s);
}

}  // namespace wtconv
