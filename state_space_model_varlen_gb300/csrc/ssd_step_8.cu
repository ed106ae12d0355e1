// Single-token step with an 8-bit state cache.
#include "ssd_step.cuh"

namespace ssd {
cudaError_t launch_step_8(const ssd_step_params &p, cudaStream_t stream) {
    return p.state_dtype == SSD_E4M3 ? launch_step_type<SSD_E4M3>(p, stream) : launch_step_type<SSD_I8>(p, stream);
}
}  // namespace ssd
