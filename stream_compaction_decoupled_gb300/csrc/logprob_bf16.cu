// logprob_bf16.cu -- token log probabilities from bf16 logits.
#include "logprob.cuh"

namespace gbs {
template cudaError_t launch_logprob<__nv_bfloat16>(const LogprobJob&, const LaunchCtx&);
template cudaError_t launch_logprob_backward<__nv_bfloat16>(const LogprobJob&, const LaunchCtx&);
}  // namespace gbs
