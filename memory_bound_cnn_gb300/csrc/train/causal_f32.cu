#include "causal.cuh"

namespace wtconv {
template cudaError_t launch_causal_forward<float>(const CausalArgs &, cudaStream_t);
template cudaError_t launch_causal_backward<float>(const CausalArgs &, cudaStream_t);
template cudaError_t launch_causal_step<float>(const CausalArgs &, void *, int, const int *, cudaStream_t);
}  // namespace wtconv
