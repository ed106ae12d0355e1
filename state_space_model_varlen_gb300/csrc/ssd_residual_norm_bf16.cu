// The residual norm of bf16 rows.
#include "ssd_residual_norm.cuh"

namespace ssd {
cudaError_t launch_residual_norm_bf16(const ssd_residual_norm_params &p, cudaStream_t stream) {
    return p.residual_dtype == SSD_F32 ? launch_norm<__nv_bfloat16, float>(p, stream)
                                       : launch_norm<__nv_bfloat16, __nv_bfloat16>(p, stream);
}
}  // namespace ssd
