// recurrence_bf16.cu -- the gated linear recurrence on bf16 values.
#include "recurrence.cuh"

namespace gbs {
template cudaError_t launch_recurrence<__nv_bfloat16>(const RecurrenceJob&, const LaunchCtx&);
template cudaError_t launch_recurrence_backward<__nv_bfloat16>(const RecurrenceJob&, const LaunchCtx&);
template cudaError_t launch_recurrence_step<__nv_bfloat16>(const RecurrenceStepJob&, const LaunchCtx&);
}  // namespace gbs
