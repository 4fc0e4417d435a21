#include "selective_fwd.cuh"

namespace wtconv {
template cudaError_t launch_selective_forward<float>(const SelectiveArgs &, cudaStream_t);
template cudaError_t launch_selective_step<float>(const SelectiveArgs &, float *, int, const int *, cudaStream_t);
}  // namespace wtconv
