// layer_norm_f16.cu -- layer norm on f16 values.
#include "layer_norm.cuh"

namespace gbs {
template cudaError_t launch_layer_norm<__half, __half>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm_backward<__half, __half>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm<__half, float>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm_backward<__half, float>(const LayerNormJob&, const LaunchCtx&);
}  // namespace gbs
