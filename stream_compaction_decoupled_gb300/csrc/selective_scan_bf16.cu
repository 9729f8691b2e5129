// selective_scan_bf16.cu -- the selective state space scan on bf16 values.
#include "selective_scan.cuh"

namespace gbs {
template cudaError_t launch_selective_scan<__nv_bfloat16>(const SelectiveScanJob&, const LaunchCtx&);
template cudaError_t launch_selective_scan_backward<__nv_bfloat16>(const SelectiveScanJob&, const LaunchCtx&);
template cudaError_t launch_selective_scan_step<__nv_bfloat16>(const SelectiveScanStepJob&, const LaunchCtx&);
}  // namespace gbs
