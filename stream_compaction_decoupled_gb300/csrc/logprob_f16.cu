// logprob_f16.cu -- token log probabilities from f16 logits.
#include "logprob.cuh"

namespace gbs {
template cudaError_t launch_logprob<__half>(const LogprobJob&, const LaunchCtx&);
template cudaError_t launch_logprob_backward<__half>(const LogprobJob&, const LaunchCtx&);
}  // namespace gbs
