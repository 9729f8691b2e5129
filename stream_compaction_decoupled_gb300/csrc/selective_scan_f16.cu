// selective_scan_f16.cu -- the selective state space scan on fp16 values.
#include "selective_scan.cuh"

namespace gbs {
template cudaError_t launch_selective_scan<__half>(const SelectiveScanJob&, const LaunchCtx&);
template cudaError_t launch_selective_scan_backward<__half>(const SelectiveScanJob&, const LaunchCtx&);
template cudaError_t launch_selective_scan_step<__half>(const SelectiveScanStepJob&, const LaunchCtx&);
}  // namespace gbs
