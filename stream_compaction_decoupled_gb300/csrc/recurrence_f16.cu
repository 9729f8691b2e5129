// recurrence_f16.cu -- the gated linear recurrence on f16 values.
#include "recurrence.cuh"

namespace gbs {
template cudaError_t launch_recurrence<__half>(const RecurrenceJob&, const LaunchCtx&);
template cudaError_t launch_recurrence_backward<__half>(const RecurrenceJob&, const LaunchCtx&);
template cudaError_t launch_recurrence_step<__half>(const RecurrenceStepJob&, const LaunchCtx&);
}  // namespace gbs
