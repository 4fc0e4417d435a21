// Arguments and launch functions of the selective scan (wtconv_ssm.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "train_common.h"
#include "wtconv_ssm.h"

namespace wtconv {

constexpr int kSelTile = 32;                     // channels of a CTA
constexpr int kSelKeep = WTCONV_SELECTIVE_KEEP;  // positions of a block of the backward
constexpr int kSelRound = 32;                    // positions of a round of the forward; segments are multiples of it

// Lanes that share a channel's states, four each: 2, 4, 8 or 16.
inline int selective_lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

struct SelectiveArgs {
    wtconv_selective_shape s;
    wtconv_selective_inputs in;
    int channels;       // of a group
    int tiles;          // of a group, kSelTile channels each (the last may have fewer)
    int lanes, padded;  // selective_lanes(N), and 4 states for each
    bool wide;          // pairs of neighbours lie at multiples of their size in every activation but B and C
    int keep;           // kept states of a sequence, ceil(T / kSelKeep)
    int segments, segment;  // parts of a sequence that different CTAs scan, and positions of each
    wtconv_ssm_tensor y, dy;
    wtconv_selective_grads g;
    float *h_last, *states_out;
    const float *states_in, *dh_last;
    // workspace
    float *ends;    // [B][segments][C][padded]: the state (backward: gradient) that a segment alone ends with
    float *steps;   // [B][segments][C]: sum of d over a segment
    float *part_bc; // [G tiles][B][T][2][padded]: dB and dC of a tile's channels
    float *part_a;  // [B][segments][C][N]: dA
    float *part_c;  // [2][B][segments][C]: dD, d_dt_bias
    __host__ __device__ int ctas() const { return s.B * s.G * tiles; }  // of one segment
};

// f(lanes, planes, wide) as constants.
template <typename F> cudaError_t with_selective_shape(const SelectiveArgs &a, F f) {
    const auto with_lanes = [&](auto planes, auto wide) {
        switch (a.lanes) {
            case 2: return f(std::integral_constant<int, 2>(), planes, wide);
            case 4: return f(std::integral_constant<int, 4>(), planes, wide);
            case 8: return f(std::integral_constant<int, 8>(), planes, wide);
            default: return f(std::integral_constant<int, 16>(), planes, wide);
        }
    };
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    const std::true_type yes;
    const std::false_type no;
    return planes ? (a.wide ? with_lanes(yes, yes) : with_lanes(yes, no)) : (a.wide ? with_lanes(no, yes) : with_lanes(no, no));
}

template <typename T> cudaError_t launch_selective_forward(const SelectiveArgs &a, cudaStream_t st);
template <typename T> cudaError_t launch_selective_backward(const SelectiveArgs &a, cudaStream_t st);
template <typename T>
cudaError_t launch_selective_step(const SelectiveArgs &a, float *pool, int n_states, const int *slots, cudaStream_t st);

}  // namespace wtconv
