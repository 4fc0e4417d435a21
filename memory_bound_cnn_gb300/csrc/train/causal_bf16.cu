#include "causal.cuh"

namespace wtconv {
template cudaError_t launch_causal_forward<__nv_bfloat16>(const CausalArgs &, cudaStream_t);
template cudaError_t launch_causal_backward<__nv_bfloat16>(const CausalArgs &, cudaStream_t);
template cudaError_t launch_causal_step<__nv_bfloat16>(const CausalArgs &, void *, int, const int *, cudaStream_t);
}  // namespace wtconv
