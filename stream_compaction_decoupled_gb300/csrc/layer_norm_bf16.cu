// layer_norm_bf16.cu -- layer norm on bf16 values.
#include "layer_norm.cuh"

namespace gbs {
template cudaError_t launch_layer_norm<__nv_bfloat16, __nv_bfloat16>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm_backward<__nv_bfloat16, __nv_bfloat16>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm<__nv_bfloat16, float>(const LayerNormJob&, const LaunchCtx&);
template cudaError_t launch_layer_norm_backward<__nv_bfloat16, float>(const LayerNormJob&, const LaunchCtx&);
}  // namespace gbs
