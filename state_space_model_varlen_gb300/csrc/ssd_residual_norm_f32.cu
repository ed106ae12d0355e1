// The residual norm of fp32 rows.
#include "ssd_residual_norm.cuh"

namespace ssd {
cudaError_t launch_residual_norm_f32(const ssd_residual_norm_params &p, cudaStream_t stream) {
    return p.residual_dtype == SSD_F32 ? launch_norm<float, float>(p, stream) : launch_norm<float, __nv_bfloat16>(p, stream);
}
}  // namespace ssd
