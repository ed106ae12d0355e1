// Single-token step with a state cache in e4m3.
#include "ssd_step.cuh"

namespace ssd {
cudaError_t launch_step_e4m3(const ssd_step_params &p, cudaStream_t stream) { return launch_step_type<SSD_E4M3>(p, stream); }
}  // namespace ssd
