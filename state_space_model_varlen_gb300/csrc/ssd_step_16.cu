// Single-token step with a 16-bit state cache.
#include "ssd_step.cuh"

namespace ssd {
cudaError_t launch_step_16(const ssd_step_params &p, cudaStream_t stream) {
    return p.state_dtype == SSD_BF16 ? launch_step_type<SSD_BF16>(p, stream) : launch_step_type<SSD_F16>(p, stream);
}
}  // namespace ssd
