#include "norm.cuh"

namespace wtconv {
template cudaError_t launch_norm_forward<__half, __half>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<__half, __half>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_forward<__half, float>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<__half, float>(const NormArgs &, cudaStream_t);
}  // namespace wtconv
