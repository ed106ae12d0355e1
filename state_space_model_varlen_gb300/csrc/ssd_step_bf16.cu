// Single-token step with a state cache in bf16.
#include "ssd_step.cuh"

namespace ssd {
cudaError_t launch_step_bf16(const ssd_step_params &p, cudaStream_t stream) { return launch_step_type<SSD_BF16>(p, stream); }
}  // namespace ssd
