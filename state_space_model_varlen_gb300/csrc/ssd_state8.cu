// States to and from an 8-bit cache: one scale per state row.
//
// Store reads a row once, takes its largest magnitude over the eight lanes
// that share it and writes codes and scale; load multiplies codes by their
// scale.  Both are bound by HBM.
#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;

// the slot of state s, or -1 (reported) where it is none
__device__ __forceinline__ int checked_slot(const ssd_state_params &a, int s, bool reporter) {
    const int slot = a.slot_idx[(int64_t)s * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
    if (slot >= 0 && slot < a.num_slots) return slot;
    if (reporter && a.device_status) atomicOr(a.device_status, SSD_DEV_BAD_SLOT);
    return -1;
}

template <typename DnT, int kType, int E, int V>
__global__ void __launch_bounds__(kThreads) store_kernel(const ssd_state_params a, int blocks) {
    const int s = blockIdx.x / blocks, N = a.dstate;
    const int64_t per = (int64_t)a.nheads * a.headdim;
    const int64_t r = (int64_t)(blockIdx.x % blocks) * kGroups + (threadIdx.x >> 3);
    const int lane8 = threadIdx.x & 7;
    __shared__ __align__(16) uint32_t keys[20];
    if (a.sr_seed && threadIdx.x < 20) round_keys(*a.sr_seed, threadIdx.x, keys);
    __syncthreads();
    const int slot = checked_slot(a, s, threadIdx.x == 0 && blockIdx.x % blocks == 0);
    if (slot < 0) return;
    const bool live = r < per;
    const DnT *src = static_cast<const DnT *>(a.states) + ((int64_t)s * per + r) * N;
    float v[E / V][V];
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
        const int n = (k * 8 + lane8) * V;
        Pack<DnT, V> p{};
        if (live && n < N) p = load_pack<DnT, V>(src + n);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[k][j] = to_float(p.v[j]);
            big = max_abs(big, v[k][j], v[k][j]);
        }
    }
    float inv, scale;
    row_scale(lanes_max<8>(big), code_limit<kType>(), &inv, &scale);
    if (!live) return;
    const int64_t row = (int64_t)slot * per + r;
    if (lane8 == 0) a.state_scale[row] = scale;
    uint8_t *dst = static_cast<uint8_t *>(a.state_cache) + row * N;
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
        const int n = (k * 8 + lane8) * V;
        if (n >= N) continue;
        store_pack<uint8_t, V>(dst + n, a.sr_seed ? encode8_sr<kType, V>(v[k], inv, keys, (uint64_t)(row * N + n))
                                                  : encode8<kType, V>(v[k], inv));
    }
}

template <typename DnT, int kType, int E, int V>
__global__ void __launch_bounds__(kThreads) load_kernel(const ssd_state_params a, int blocks) {
    const int s = blockIdx.x / blocks, N = a.dstate;
    const int64_t per = (int64_t)a.nheads * a.headdim;
    const int64_t r = (int64_t)(blockIdx.x % blocks) * kGroups + (threadIdx.x >> 3);
    const int lane8 = threadIdx.x & 7;
    const bool init = a.has_init == nullptr || a.has_init[s] != 0;
    int slot = 0;
    if (init) {
        slot = checked_slot(a, s, threadIdx.x == 0 && blockIdx.x % blocks == 0);
        if (slot < 0) return;
    }
    if (r >= per) return;
    const int64_t row = (int64_t)slot * per + r;
    const float scale = init ? a.state_scale[row] : 0.f;
    const uint8_t *src = static_cast<const uint8_t *>(a.state_cache) + row * N;
    DnT *dst = static_cast<DnT *>(a.states) + ((int64_t)s * per + r) * N;
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
        const int n = (k * 8 + lane8) * V;
        if (n >= N) continue;
        float v[V];
        Pack<DnT, V> out;
        if (init) decode<kType, V>(load_pack<uint8_t, V>(src + n), v);
#pragma unroll
        for (int j = 0; j < V; ++j) out.v[j] = from_float<DnT>(init ? v[j] * scale : 0.f);
        store_pack<DnT, V>(dst + n, out);
    }
}

template <bool kStore, typename DnT, int kType, int E, int V>
cudaError_t launch(const ssd_state_params &p, cudaStream_t stream) {
    const int64_t per = (int64_t)p.nheads * p.headdim, blocks = (per + kGroups - 1) / kGroups;
    if (p.num_states * blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)(p.num_states * blocks);
    if (kStore) store_kernel<DnT, kType, E, V><<<grid, kThreads, 0, stream>>>(p, (int)blocks);
    else load_kernel<DnT, kType, E, V><<<grid, kThreads, 0, stream>>>(p, (int)blocks);
    return cudaGetLastError();
}

template <bool kStore, typename DnT, int kType>
cudaError_t launch_n(const ssd_state_params &p, cudaStream_t stream) {
    const int io = (int)sizeof(DnT);
    const bool four = p.dstate % 4 == 0 && aligned_to(p.state_cache, 4) && aligned_to(p.states, 4 * io);
    if (four) {
        if (p.dstate <= 64) return launch<kStore, DnT, kType, 8, 4>(p, stream);
        if (p.dstate <= 128) return launch<kStore, DnT, kType, 16, 4>(p, stream);
        return launch<kStore, DnT, kType, 32, 4>(p, stream);
    }
    if (p.dstate <= 64) return launch<kStore, DnT, kType, 8, 1>(p, stream);
    if (p.dstate <= 128) return launch<kStore, DnT, kType, 16, 1>(p, stream);
    return launch<kStore, DnT, kType, 32, 1>(p, stream);
}

template <bool kStore>
cudaError_t launch_any(const ssd_state_params &p, cudaStream_t stream) {
    if (p.dense_dtype == SSD_F32)
        return p.state_dtype == SSD_E4M3 ? launch_n<kStore, float, SSD_E4M3>(p, stream)
                                         : launch_n<kStore, float, SSD_I8>(p, stream);
    return p.state_dtype == SSD_E4M3 ? launch_n<kStore, __nv_bfloat16, SSD_E4M3>(p, stream)
                                     : launch_n<kStore, __nv_bfloat16, SSD_I8>(p, stream);
}

}  // namespace

cudaError_t launch_state_store(const ssd_state_params &p, cudaStream_t stream) { return launch_any<true>(p, stream); }
cudaError_t launch_state_load(const ssd_state_params &p, cudaStream_t stream) { return launch_any<false>(p, stream); }

}  // namespace ssd
