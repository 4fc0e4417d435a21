#include "selective_bwd.cuh"

namespace wtconv {
template cudaError_t launch_selective_backward<__half>(const SelectiveArgs &, cudaStream_t);
}  // namespace wtconv
