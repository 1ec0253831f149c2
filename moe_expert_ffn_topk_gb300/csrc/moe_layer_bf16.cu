// moe_layer's kernels for one weight format.
#include "moe_layer.cuh"

namespace moe {
namespace layer {
template cudaError_t launch_fmt<MOE_LAYER_BF16>(const Args&, cudaStream_t);
}  // namespace layer
}  // namespace moe
