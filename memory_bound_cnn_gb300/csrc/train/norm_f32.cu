#include "norm.cuh"

namespace wtconv {
template cudaError_t launch_norm_forward<float, float>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<float, float>(const NormArgs &, cudaStream_t);
}  // namespace wtconv
