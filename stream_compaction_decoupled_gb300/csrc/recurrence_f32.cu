// recurrence_f32.cu -- the gated linear recurrence on f32 values.
#include "recurrence.cuh"

namespace gbs {
template cudaError_t launch_recurrence<float>(const RecurrenceJob&, const LaunchCtx&);
template cudaError_t launch_recurrence_backward<float>(const RecurrenceJob&, const LaunchCtx&);
template cudaError_t launch_recurrence_step<float>(const RecurrenceStepJob&, const LaunchCtx&);
}  // namespace gbs
