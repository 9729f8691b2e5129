// verify_drafts_f32.cu -- the verification of drafted tokens with fp32 probabilities.
#include "verify_drafts.cuh"

namespace gbs {
template cudaError_t launch_verify<float>(const VerifyJob&, const LaunchCtx&);
}  // namespace gbs
