// logprob_f32.cu -- token log probabilities from f32 logits.
#include "logprob.cuh"

namespace gbs {
template cudaError_t launch_logprob<float>(const LogprobJob&, const LaunchCtx&);
template cudaError_t launch_logprob_backward<float>(const LogprobJob&, const LaunchCtx&);
}  // namespace gbs
