// selective_scan_f32.cu -- the selective state space scan on fp32 values.
#include "selective_scan.cuh"

namespace gbs {
template cudaError_t launch_selective_scan<float>(const SelectiveScanJob&, const LaunchCtx&);
template cudaError_t launch_selective_scan_backward<float>(const SelectiveScanJob&, const LaunchCtx&);
template cudaError_t launch_selective_scan_step<float>(const SelectiveScanStepJob&, const LaunchCtx&);
}  // namespace gbs
