#include "norm.cuh"

namespace wtconv {
template cudaError_t launch_norm_forward<__nv_bfloat16, __nv_bfloat16>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<__nv_bfloat16, __nv_bfloat16>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_forward<__nv_bfloat16, float>(const NormArgs &, cudaStream_t);
template cudaError_t launch_norm_backward<__nv_bfloat16, float>(const NormArgs &, cudaStream_t);
}  // namespace wtconv
