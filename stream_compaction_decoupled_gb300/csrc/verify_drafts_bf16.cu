// verify_drafts_bf16.cu -- the verification of drafted tokens with bf16 probabilities.
#include "verify_drafts.cuh"

namespace gbs {
template cudaError_t launch_verify<__nv_bfloat16>(const VerifyJob&, const LaunchCtx&);
}  // namespace gbs
