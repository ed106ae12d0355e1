// Internal declarations of the layer operators' translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd_layer.h"
#include "ssd_mixer_internal.h"

namespace ssd {

// Each launches exactly one kernel; the arguments have been checked.
cudaError_t launch_residual_norm_f32(const ssd_residual_norm_params &p, cudaStream_t stream);
cudaError_t launch_residual_norm_bf16(const ssd_residual_norm_params &p, cudaStream_t stream);
cudaError_t launch_matvec4(const ssd_matvec4_params &p, cudaStream_t stream);
cudaError_t launch_verify(const ssd_verify_params &p, cudaStream_t stream);

// enqueue() with dynamic shared memory (at most 48 KB with the arrays that the kernel declares itself)
template <typename... Params, typename... Args>
cudaError_t enqueue_shared(void (*kernel)(Params...), dim3 grid, int threads, size_t shared, cudaStream_t stream,
                           const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3((unsigned)threads);
    config.dynamicSmemBytes = shared;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, Params(args)...);
}

}  // namespace ssd
