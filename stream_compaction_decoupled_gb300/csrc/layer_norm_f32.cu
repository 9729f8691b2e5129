// layer_norm_f32.cu -- layer norm on f32 values.
#include "layer_norm.cuh"

namespace gbs {
template cudaError_t launch_layer_norm<float, float>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm_backward<float, float>(const LayerNormJob&, const LaunchCtx&);
}  // namespace gbs
