#include "selective_bwd.cuh"

namespace wtconv {
template cudaError_t launch_selective_backward<float>(const SelectiveArgs &, cudaStream_t);
}  // namespace wtconv
