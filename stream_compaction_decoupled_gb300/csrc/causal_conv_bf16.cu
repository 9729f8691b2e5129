// causal_conv_bf16.cu -- the causal convolution on bf16 values.
#include "causal_conv.cuh"

namespace gbs {
template cudaError_t launch_causal_conv<__nv_bfloat16>(const CausalConvJob&, const LaunchCtx&);
template cudaError_t launch_causal_conv_backward<__nv_bfloat16>(const CausalConvJob&, const LaunchCtx&);
template cudaError_t launch_causal_conv_step<__nv_bfloat16>(const CausalConvStepJob&, const LaunchCtx&);
}  // namespace gbs
