// Internal declarations of the mixer operators' translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd_mixer.h"

namespace ssd {

// Each launches exactly one kernel; the arguments have been checked.
cudaError_t launch_conv(const ssd_conv_params &p, cudaStream_t stream);
cudaError_t launch_gated_norm(const ssd_gated_norm_params &p, cudaStream_t stream);
cudaError_t launch_state_store(const ssd_state_params &p, cudaStream_t stream);
cudaError_t launch_state_load(const ssd_state_params &p, cudaStream_t stream);
// The step, one translation unit for each type of the state cache.
cudaError_t launch_step_f32(const ssd_step_params &p, cudaStream_t stream);
cudaError_t launch_step_bf16(const ssd_step_params &p, cudaStream_t stream);
cudaError_t launch_step_f16(const ssd_step_params &p, cudaStream_t stream);
cudaError_t launch_step_e4m3(const ssd_step_params &p, cudaStream_t stream);
cudaError_t launch_step_i8(const ssd_step_params &p, cudaStream_t stream);

// Every kernel of these operators is launched so that it may be set up while
// the kernel before it in the stream drains (programmatic dependent launch),
// and starts with await_previous().  Store and load of three states back to
// back: 8.6 us so, 12.2 with plain launches.
template <typename... Params, typename... Args>
cudaError_t enqueue(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3((unsigned)threads);
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, Params(args)...);
}

inline bool aligned_to(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

// The widest vector of a state row, in elements of `size` bytes: 16 bytes
// where the row's bytes and the base allow it, then 4 elements, then 1.
// `lanes` lanes share a row, so rows of fewer vectors take narrower ones.
inline int state_vector(int n, int size, const void *base, int lanes) {
    for (int v : {16 / size, 4})
        if (v >= 4 && n % v == 0 && (n / v >= lanes || v == 4) && aligned_to(base, (size_t)v * size)) return v;
    return 1;
}

}  // namespace ssd
