#include "causal.cuh"

namespace wtconv {
template cudaError_t launch_causal_forward<__half>(const CausalArgs &, cudaStream_t);
template cudaError_t launch_causal_backward<__half>(const CausalArgs &, cudaStream_t);
template cudaError_t launch_causal_step<__half>(const CausalArgs &, void *, int, const int *, cudaStream_t);
}  // namespace wtconv
