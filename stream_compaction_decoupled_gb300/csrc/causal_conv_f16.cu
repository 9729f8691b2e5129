// causal_conv_f16.cu -- the causal convolution on fp16 values.
#include "causal_conv.cuh"

namespace gbs {
template cudaError_t launch_causal_conv<__half>(const CausalConvJob&, const LaunchCtx&);
template cudaError_t launch_causal_conv_backward<__half>(const CausalConvJob&, const LaunchCtx&);
template cudaError_t launch_causal_conv_step<__half>(const CausalConvStepJob&, const LaunchCtx&);
}  // namespace gbs
