// Single-token step of a Mamba2 mixer: convolution, dt, state update, read-out
// and gate of one token per request, in one launch.
//
//   u = act(bias + sum_k w[:, W-1-k] xbc_{pos-k}),   u = (x, B, C)
//   h <- exp(dt' A) h + dt' x B^T,   y = (C h + D x) SiLU(z)
//
// The state is read once and written once and dwarfs the rest (N values for
// each x): the kernel is bound by HBM, for small batches by latency.  One CTA
// takes a request's head, or a block of its rows.  Eight lanes share a state
// row, so that a row's sums and maxima take three shuffles, and a warp's four
// rows are neighbours in memory.  Every thread issues the loads of all its
// rows before the convolution, which needs the same indices: one memory round
// trip covers both.
//
// The convolution cache is a ring, so the row the call writes (pos mod rows)
// is none of those its other CTAs read, and they need no order among them.
// Every CTA of a group convolves the group's B and C for itself (from L2).
#pragma once

#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kStepThreads = 128;
constexpr int kStepGroups = kStepThreads / 8;      // state rows in flight at a time

// One channel's convolution at position pos; the newest input is `now`.
template <typename IoT>
__device__ __forceinline__ float conv_channel(const ssd_step_params &a, const IoT *xbc, const IoT *ring, int channels,
                                              int c, int pos, int row) {
    const IoT *w = static_cast<const IoT *>(a.weight) + (int64_t)c * a.width;
    float acc = a.bias ? to_float(static_cast<const IoT *>(a.bias)[c]) : 0.f;
    acc = fmaf(to_float(w[a.width - 1]), to_float(xbc[c]), acc);
#pragma unroll
    for (int k = 1; k < SSD_CONV_MAX_WIDTH; ++k) {
        if (k < a.width && k <= pos) {
            int r = row - k;
            if (r < 0) r += a.conv_rows;
            acc = fmaf(to_float(w[a.width - 1 - k]), to_float(ring[(int64_t)r * channels + c]), acc);
        }
    }
    return a.activation ? silu(acc) : acc;
}

// kType: storage of the state; E: state values a lane holds of a row (8 E >=
// N); V: values of one load.  kRows: rows a lane works on.
template <int kType, int E, int V, int kRows>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const ssd_step_params a, int row_blocks) {
    using StT = typename Stored<kType>::T;
    constexpr int kTile = kStepGroups * kRows;
    constexpr int kChunks = E / V;
    constexpr bool k8bit = kType == SSD_E4M3 || kType == SSD_I8;
    __shared__ float s_b[8 * E], s_c[8 * E], s_x[kTile], s_y[kTile], s_dt[2];

    const int N = a.dstate, P = a.headdim, H = a.nheads;
    const int pb = blockIdx.x % row_blocks;
    const int h = (blockIdx.x / row_blocks) % H;
    const int b = blockIdx.x / row_blocks / H;
    const int tid = threadIdx.x, lane8 = tid & 7, grp = tid >> 3;
    const int p0 = pb * kTile, rows = min(kTile, P - p0);
    const int64_t yrow = ((int64_t)b * H + h) * P + p0;
    const bool bf16 = a.io_dtype == SSD_BF16;

    const int slot = a.slot_idx[(int64_t)b * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
    const int pos = a.pos[b];
    if (slot < 0 || slot >= a.num_slots || pos < 0) {
        if (slot == -1) {
            for (int i = tid; i < rows; i += kStepThreads) {
                if (bf16) static_cast<__nv_bfloat16 *>(a.out_y)[yrow + i] = __float2bfloat16_rn(0.f);
                else static_cast<float *>(a.out_y)[yrow + i] = 0.f;
            }
        } else if (tid == 0 && pb == 0 && h == 0 && a.device_status) {
            atomicOr(a.device_status, pos < 0 ? SSD_DEV_BAD_POS : SSD_DEV_BAD_SLOT);
        }
        return;
    }

    // ---- the state's loads -------------------------------------------------
    const int64_t row0 = ((int64_t)slot * H + h) * P + p0;         // row of the cache
    StT *cache = static_cast<StT *>(a.state_cache) + row0 * N;
    Pack<StT, V> raw[kRows][kChunks];
    float scale[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = grp + i * kStepGroups;
        scale[i] = 0.f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const int n = (k * 8 + lane8) * V;
            raw[i][k] = Pack<StT, V>{};
            if (r < rows && n < N && pos > 0) raw[i][k] = load_pack<StT, V>(cache + (int64_t)r * N + n);
        }
        if (k8bit && r < rows && pos > 0) scale[i] = a.state_scale[row0 + r];
    }

    // ---- convolution -------------------------------------------------------
    const int channels = H * P + 2 * a.ngroups * N;
    const int g = h / (H / a.ngroups);
    const int ring_row = pos % a.conv_rows;
    const bool writes_bc = pb == 0 && h % (H / a.ngroups) == 0;
    auto convolve = [&](auto io) {
        using IoT = decltype(io);
        const IoT *xbc = static_cast<const IoT *>(a.xbc) + (int64_t)b * a.xbc_stride;
        IoT *ring = static_cast<IoT *>(a.conv_cache) + (int64_t)slot * a.conv_rows * channels;
        for (int i = tid; i < 2 * N + rows; i += kStepThreads) {
            int c;
            float *dst;
            if (i < N) {
                c = H * P + g * N + i;
                dst = s_b + i;
            } else if (i < 2 * N) {
                c = H * P + (a.ngroups + g) * N + (i - N);
                dst = s_c + (i - N);
            } else {
                c = h * P + p0 + (i - 2 * N);
                dst = s_x + (i - 2 * N);
            }
            *dst = conv_channel<IoT>(a, xbc, ring, channels, c, pos, ring_row);
            if (i >= 2 * N || writes_bc) ring[(int64_t)ring_row * channels + c] = xbc[c];
        }
        if (tid == 0) {
            float dt = to_float(static_cast<const IoT *>(a.dt)[(int64_t)b * a.dt_stride + h]);
            if (a.dt_bias) dt += a.dt_bias[h];
            if (a.dt_softplus) dt = softplus(dt);
            s_dt[0] = dt;
            s_dt[1] = expf(dt * a.A[h]);
        }
    };
    for (int i = tid; i < 8 * E; i += kStepThreads)
        if (i >= N) s_b[i] = s_c[i] = 0.f;
    if (bf16) convolve(__nv_bfloat16{});
    else convolve(float{});
    __syncthreads();

    // ---- update and read-out -----------------------------------------------
    const float dt = s_dt[0], decay = s_dt[1];
    float bv[E], cv[E];
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            bv[k * V + j] = s_b[(k * 8 + lane8) * V + j];
            cv[k * V + j] = s_c[(k * 8 + lane8) * V + j];
        }
    const uint64_t seed = a.sr_seed ? *a.sr_seed : 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = grp + i * kStepGroups;
        const float dx = r < rows ? dt * s_x[r] : 0.f;
        const float keep = k8bit ? decay * scale[i] : decay;
        float st[kChunks][V];
        float acc = 0.f;
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            decode<kType, V>(raw[i][k], st[k]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                st[k][j] = fmaf(keep, st[k][j], dx * bv[k * V + j]);
                acc = fmaf(cv[k * V + j], st[k][j], acc);
                if (k8bit) big = max(big, __float_as_uint(st[k][j]) & 0x7fffffffu);
            }
        }
        acc = sum8(acc);
        if (lane8 == 0 && r < rows) s_y[r] = acc;
        float inv = 0.f, sc = 0.f;
        if constexpr (k8bit) {
            row_scale(max8(big), code_limit<kType>(), &inv, &sc);
            if (lane8 == 0 && r < rows) a.state_scale[row0 + r] = sc;
        }
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const int n = (k * 8 + lane8) * V;
            if (r >= rows || n >= N) continue;
            StT *dst = cache + (int64_t)r * N + n;
            const uint64_t e = (uint64_t)(row0 + r) * N + n;
            Pack<StT, V> p;
            if constexpr (kType == SSD_F32) {
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = st[k][j];
            } else if constexpr (kType == SSD_BF16) {
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = __float2bfloat16_rn(st[k][j]);
            } else if constexpr (kType == SSD_F16) {
                uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (a.sr_seed) {
                        if (j == 0 || ((e + j) & 3) == 0) w = sr_block(seed, (e + j) >> 2, 0u);
                        p.v[j] = sr_f16(st[k][j], sr_word(w, (uint32_t)(e + j) & 3u));
                    } else {
                        p.v[j] = __float2half_rn(st[k][j]);
                    }
                }
            } else {
                p = a.sr_seed ? encode8_sr<kType, V>(st[k], inv, seed, e) : encode8<kType, V>(st[k], inv);
            }
            store_pack<StT, V>(dst, p);
        }
    }
    __syncthreads();

    // ---- y ------------------------------------------------------------------
    for (int i = tid; i < rows; i += kStepThreads) {
        float y = s_y[i] + (a.D ? a.D[h] * s_x[i] : 0.f);
        if (bf16) {
            if (a.z) y *= silu(__bfloat162float(static_cast<const __nv_bfloat16 *>(a.z)[(int64_t)b * a.z_stride + h * P + p0 + i]));
            static_cast<__nv_bfloat16 *>(a.out_y)[yrow + i] = __float2bfloat16_rn(y);
        } else {
            if (a.z) y *= silu(static_cast<const float *>(a.z)[(int64_t)b * a.z_stride + h * P + p0 + i]);
            static_cast<float *>(a.out_y)[yrow + i] = y;
        }
    }
}

template <int kType, int E, int V>
cudaError_t launch_step(const ssd_step_params &p, cudaStream_t stream) {
    // a lane's raw state values: 4 rows, or 2 where they would take 512 bytes
    constexpr int kRows = E * (int)sizeof(typename Stored<kType>::T) > 64 ? 2 : 4;
    const int row_blocks = (p.headdim + kStepGroups * kRows - 1) / (kStepGroups * kRows);
    const int64_t grid = (int64_t)p.batch * p.nheads * row_blocks;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    step_kernel<kType, E, V, kRows><<<(unsigned)grid, kStepThreads, 0, stream>>>(p, row_blocks);
    return cudaGetLastError();
}

template <int kType, int E>
cudaError_t launch_step_vec(const ssd_step_params &p, cudaStream_t stream) {
    constexpr int size = (int)sizeof(typename Stored<kType>::T);
    const int v = state_vector(p.dstate, size, p.state_cache);
    if constexpr (16 / size <= E) if (v == 16 / size) return launch_step<kType, E, 16 / size>(p, stream);
    if constexpr (8 / size >= 4 && 8 / size <= E) if (v == 8 / size) return launch_step<kType, E, 8 / size>(p, stream);
    if constexpr (4 <= E) if (v == 4) return launch_step<kType, E, 4>(p, stream);
    return launch_step<kType, E, 1>(p, stream);
}

template <int kType>
cudaError_t launch_step_type(const ssd_step_params &p, cudaStream_t stream) {
    if (p.dstate <= 64) return launch_step_vec<kType, 8>(p, stream);
    if (p.dstate <= 128) return launch_step_vec<kType, 16>(p, stream);
    return launch_step_vec<kType, 32>(p, stream);
}

}  // namespace
}  // namespace ssd
