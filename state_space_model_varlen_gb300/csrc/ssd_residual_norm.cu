// Residual addition and RMS norm, with an output in 8 bits.
//
//   v = x + residual;  n = v / sqrt(mean(v^2) + eps) weight;  codes of n by groups
//
// Each value is read once and written once: bound by HBM.
#include "ssd_layer_internal.h"
#include "ssd_mixer_common.cuh"

namespace ssd {
namespace {

__device__ __forceinline__ float warp_sum(float v) { return lanes_sum<32>(v); }
// over the CTA, whose warps leave their sums in part
__device__ __forceinline__ float cta_sum(float v, float *part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < blockDim.x / 32 ? part[threadIdx.x & 31] : 0.f;
    return warp_sum(v);
}

// one row
template <typename IoT, typename ResT> struct Row {
    const IoT *x, *w;
    const ResT *res;
    ResT *res_out;
    IoT *out;
    uint8_t *codes;
    float *scale;
    __device__ Row(const ssd_residual_norm_params &a, int64_t row) {
        x = static_cast<const IoT *>(a.x) + row * a.x_stride;
        w = static_cast<const IoT *>(a.weight);
        res = a.residual ? static_cast<const ResT *>(a.residual) + row * a.residual_stride : nullptr;
        res_out = a.residual_out ? static_cast<ResT *>(a.residual_out) + row * a.residual_out_stride : nullptr;
        out = a.out ? static_cast<IoT *>(a.out) + row * a.out_stride : nullptr;
        codes = a.out_codes ? a.out_codes + row * a.codes_stride : nullptr;
        scale = a.out_codes ? a.out_scale + row * (a.columns / a.scale_group) : nullptr;
    }
    __device__ float sum(int c) const {
        float v = to_float(x[c]);
        if (res) v += to_float(res[c]);
        return v;
    }
    __device__ float normed(float v, float r, int c) const { return w ? v * r * to_float(w[c]) : v * r; }
    __device__ void store(int c, float v, float n) const {
        if (res_out) res_out[c] = from_float<ResT>(v);
        if (out) out[c] = from_float<IoT>(n);
    }
};

// Rows that no other variant takes: a CTA a row, element by element, read again
// for the norm and again for the codes, whose groups go to a warp each (a value is
// written by the thread that read it last).
template <typename IoT, typename ResT>
__global__ void __launch_bounds__(1024) residual_norm_any_kernel(const ssd_residual_norm_params a) {
    __shared__ float part[32];
    await_previous();
    const Row<IoT, ResT> row(a, blockIdx.x);
    float two = 0.f;
    for (int c = threadIdx.x; c < a.columns; c += blockDim.x) {
        const float v = row.sum(c);
        two = fmaf(v, v, two);
    }
    const float r = 1.f / sqrtf(cta_sum(two, part) / (float)a.columns + a.eps);
    if (!row.codes) {
        for (int c = threadIdx.x; c < a.columns; c += blockDim.x) {
            const float v = row.sum(c);
            row.store(c, v, row.normed(v, r, c));
        }
        return;
    }
    const int lane = threadIdx.x & 31, G = a.scale_group;
    for (int g = threadIdx.x >> 5; g < a.columns / G; g += blockDim.x >> 5) {
        float m = 0.f;
        for (int c = lane; c < G; c += 32) {
            const float n = row.normed(row.sum(g * G + c), r, g * G + c);
            m = max_abs(m, n, n);
        }
        m = lanes_max<32>(m);
        float inv, scale;
        row_scale(m, a.code_dtype == SSD_E4M3 ? code_limit<SSD_E4M3>() : code_limit<SSD_I8>(), &inv, &scale);
        if (lane == 0) row.scale[g] = scale;
        for (int i = lane; i < G; i += 32) {
            const int c = g * G + i;
            const float v = row.sum(c), n = row.normed(v, r, c);
            row.store(c, v, n);
            row.codes[c] = a.code_dtype == SSD_E4M3 ? encode1<SSD_E4M3>(n, inv) : encode1<SSD_I8>(n, inv);
        }
    }
}

template <typename IoT, typename ResT> cudaError_t launch(const ssd_residual_norm_params &p, cudaStream_t stream) {
    if (p.rows > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int threads = p.columns >= 1024 ? 1024 : (p.columns + 31) / 32 * 32;
    return enqueue(residual_norm_any_kernel<IoT, ResT>, dim3((unsigned)p.rows), threads, stream, p);
}

}  // namespace

cudaError_t launch_residual_norm(const ssd_residual_norm_params &p, cudaStream_t stream) {
    const bool wide = p.residual_dtype == SSD_F32;
    if (p.io_dtype == SSD_F32) return wide ? launch<float, float>(p, stream) : launch<float, __nv_bfloat16>(p, stream);
    return wide ? launch<__nv_bfloat16, float>(p, stream) : launch<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace ssd
