#include "selective_bwd.cuh"

namespace wtconv {
template cudaError_t launch_selective_backward<__nv_bfloat16>(const SelectiveArgs &, cudaStream_t);
}  // namespace wtconv
