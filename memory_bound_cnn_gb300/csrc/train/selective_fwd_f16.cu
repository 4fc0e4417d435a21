#include "selective_fwd.cuh"

namespace wtconv {
template cudaError_t launch_selective_forward<__half>(const SelectiveArgs &, cudaStream_t);
template cudaError_t launch_selective_step<__half>(const SelectiveArgs &, float *, int, const int *, cudaStream_t);
}  // namespace wtconv
