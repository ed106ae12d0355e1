// Gated RMS norm over groups of columns.
//
//   out = rms(y SiLU(z)) w   or   rms(y) w SiLU(z)
//
// Each value is read once and written once: bound by HBM.  One CTA takes one
// group of one row and keeps its values in registers between the sum of
// squares and the scaling.
#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

template <typename IoT, int V>
__global__ void __launch_bounds__(256) gated_norm_kernel(const ssd_gated_norm_params a, int groups) {
    __shared__ float part[8];
    const int64_t row = blockIdx.x / groups;
    const int c0 = (int)(blockIdx.x % groups) * a.group_size;
    const IoT *y = static_cast<const IoT *>(a.y) + row * a.y_stride + c0;
    const IoT *z = a.z ? static_cast<const IoT *>(a.z) + row * a.z_stride + c0 : nullptr;
    const IoT *w = a.weight ? static_cast<const IoT *>(a.weight) + c0 : nullptr;
    IoT *out = static_cast<IoT *>(a.out) + row * a.out_stride + c0;
    auto value = [&](int c, float (&v)[V], float (&gate)[V]) {
        const Pack<IoT, V> py = load_pack<IoT, V>(y + c);
        Pack<IoT, V> pz;
        if (z) pz = load_pack<IoT, V>(z + c);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[j] = to_float(py.v[j]);
            gate[j] = z ? silu(to_float(pz.v[j])) : 1.f;
            if (!a.norm_before_gate) {
                v[j] *= gate[j];
                gate[j] = 1.f;
            }
        }
    };
    float sum = 0.f;
    for (int c = threadIdx.x * V; c < a.group_size; c += blockDim.x * V) {
        float v[V], gate[V];
        value(c, v, gate);
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) sum += part[i];
    const float r = 1.f / sqrtf(sum / (float)a.group_size + a.eps);
    for (int c = threadIdx.x * V; c < a.group_size; c += blockDim.x * V) {
        float v[V], gate[V];
        value(c, v, gate);
        Pack<IoT, V> po;
#pragma unroll
        for (int j = 0; j < V; ++j)
            po.v[j] = from_float<IoT>(v[j] * r * (w ? to_float(w[c + j]) : 1.f) * gate[j]);
        store_pack<IoT, V>(out + c, po);
    }
}

template <typename IoT, int V>
cudaError_t launch(const ssd_gated_norm_params &p, cudaStream_t stream) {
    const int groups = p.columns / p.group_size;
    if (p.rows * groups > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    gated_norm_kernel<IoT, V><<<(unsigned)(p.rows * groups), 256, 0, stream>>>(p, groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_norm(const ssd_gated_norm_params &p, cudaStream_t stream) {
    const int io = p.io_dtype == SSD_F32 ? 4 : 2, v = 16 / io;
    const bool wide = p.group_size % v == 0 && p.y_stride % v == 0 && p.out_stride % v == 0 && p.z_stride % v == 0 &&
                      aligned_to(p.y, 16) && aligned_to(p.z, 16) && aligned_to(p.out, 16);
    if (p.io_dtype == SSD_F32) return wide ? launch<float, 4>(p, stream) : launch<float, 1>(p, stream);
    return wide ? launch<__nv_bfloat16, 8>(p, stream) : launch<__nv_bfloat16, 1>(p, stream);
}

}  // namespace ssd
