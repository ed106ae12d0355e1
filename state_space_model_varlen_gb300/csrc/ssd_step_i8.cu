// Single-token step with a state cache in int8.
#include "ssd_step.cuh"

namespace ssd {
cudaError_t launch_step_i8(const ssd_step_params &p, cudaStream_t stream) { return launch_step_type<SSD_I8>(p, stream); }
}  // namespace ssd
