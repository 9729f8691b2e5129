// verify_drafts_f16.cu -- the verification of drafted tokens with fp16 probabilities.
#include "verify_drafts.cuh"

namespace gbs {
template cudaError_t launch_verify<__half>(const VerifyJob&, const LaunchCtx&);
}  // namespace gbs
