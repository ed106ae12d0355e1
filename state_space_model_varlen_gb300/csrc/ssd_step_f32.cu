// Single-token step with a state cache in fp32.
#include "ssd_step.cuh"

namespace ssd {
cudaError_t launch_step_f32(const ssd_step_params &p, cudaStream_t stream) { return launch_step_type<SSD_F32>(p, stream); }
}  // namespace ssd
