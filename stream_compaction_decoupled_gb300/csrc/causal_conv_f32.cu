// causal_conv_f32.cu -- the causal convolution on fp32 values.
#include "causal_conv.cuh"

namespace gbs {
template cudaError_t launch_causal_conv<float>(const CausalConvJob&, const LaunchCtx&);
template cudaError_t launch_causal_conv_backward<float>(const CausalConvJob&, const LaunchCtx&);
template cudaError_t launch_causal_conv_step<float>(const CausalConvStepJob&, const LaunchCtx&);
}  // namespace gbs
