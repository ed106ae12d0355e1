// States to and from an 8-bit cache: one scale per state row.
//
// Store reads a row once, takes its largest magnitude over the eight lanes
// that share it and writes codes and scale; load multiplies codes by their
// scale.  Both are bound by HBM: 32 bf16 states of 2^20 values to e4m3 and back
// take 31.4 us, 6.5 TB/s (96 % of the copy rate).  A thread has its share of
// kRows rows, all loads of which are issued together.
#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;
constexpr int kRows = 2;                        // rows of a thread
constexpr int kTile = kGroups * kRows;          // rows of a CTA

// the slot of state s, or -1 (reported) where it is none
__device__ __forceinline__ int checked_slot(const ssd_state_params &a, int s, bool reporter) {
    const int slot = a.slot_idx[(int64_t)s * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
    if (slot >= 0 && slot < a.num_slots) return slot;
    if (reporter && a.device_status) atomicOr(a.device_status, SSD_DEV_BAD_SLOT);
    return -1;
}

template <typename DnT, int kType, int E, int V, bool kSr>
__global__ void __launch_bounds__(kThreads) store_kernel(const ssd_state_params a, int blocks) {
    __shared__ __align__(16) uint32_t keys[20];
    __shared__ uint4 s_rand[kSr ? kGroups * rand_blocks(8 * E) : 1];
    await_previous();
    const int s = blockIdx.x / blocks, N = a.dstate;
    const int64_t per = (int64_t)a.nheads * a.headdim;
    const int64_t r0 = (int64_t)(blockIdx.x % blocks) * kTile + (threadIdx.x >> 3);
    const int lane = threadIdx.x & 7;
    Pack<DnT, V> p[kRows][E / V];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int n = (k * 8 + lane) * V;
            const int64_t r = r0 + i * kGroups;
            p[i][k] = Pack<DnT, V>{};
            if (r < per && n < N)
                p[i][k] = load_pack<DnT, V>(static_cast<const DnT *>(a.states) + ((int64_t)s * per + r) * N + n);
        }
    if (kSr && threadIdx.x < 20) round_keys(*a.sr_seed, threadIdx.x, keys);
    const int slot = checked_slot(a, s, threadIdx.x == 0 && blockIdx.x % blocks == 0);
    if (slot < 0) return;
    if constexpr (kSr) __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i * kGroups, row = (int64_t)slot * per + r;
        float v[E / V][V], big = 0.f;
#pragma unroll
        for (int k = 0; k < E / V; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[k][j] = to_float(p[i][k].v[j]);
                if (j & 1) big = max_abs(big, v[k][j - 1], v[k][j]);
                else if (V == 1) big = max_abs(big, v[k][j], v[k][j]);
            }
        float inv, scale;
        row_scale(lanes_max<8>(big), code_limit<kType>(), &inv, &scale);
        uint4 *rand = s_rand + (kSr ? (threadIdx.x >> 3) * rand_blocks(8 * E) : 0);
        if constexpr (kSr) row_bytes<8>(rand, keys, (uint64_t)row * N, N, lane);
        if (r >= per) continue;
        if (lane == 0) a.state_scale[row] = scale;
        uint8_t *dst = static_cast<uint8_t *>(a.state_cache) + row * N;
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int n = (k * 8 + lane) * V;
            if (n >= N) continue;
            const uint8_t *bytes = reinterpret_cast<const uint8_t *>(rand) + (row * N & 15) + n;
            if constexpr (kSr)
                store_pack<uint8_t, V>(dst + n, encode8_sr<kType, V>(v[k], inv, keys, (uint64_t)(row * N + n), bytes));
            else
                store_pack<uint8_t, V>(dst + n, encode8<kType, V>(v[k], inv));
        }
    }
}

template <typename DnT, int kType, int E, int V>
__global__ void __launch_bounds__(kThreads) load_kernel(const ssd_state_params a, int blocks) {
    await_previous();
    const int s = blockIdx.x / blocks, N = a.dstate;
    const int64_t per = (int64_t)a.nheads * a.headdim;
    const int64_t r0 = (int64_t)(blockIdx.x % blocks) * kTile + (threadIdx.x >> 3);
    const int lane = threadIdx.x & 7;
    const bool init = a.has_init == nullptr || a.has_init[s] != 0;
    int slot = 0;
    if (init) {
        slot = checked_slot(a, s, threadIdx.x == 0 && blockIdx.x % blocks == 0);
        if (slot < 0) return;
    }
    Pack<uint8_t, V> p[kRows][E / V];
    float scale[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i * kGroups, row = (int64_t)slot * per + r;
        const bool live = init && r < per;
        scale[i] = live ? a.state_scale[row] : 0.f;
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int n = (k * 8 + lane) * V;
            p[i][k] = Pack<uint8_t, V>{};
            if (live && n < N) p[i][k] = load_pack<uint8_t, V>(static_cast<const uint8_t *>(a.state_cache) + row * N + n);
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i * kGroups;
        DnT *dst = static_cast<DnT *>(a.states) + ((int64_t)s * per + r) * N;
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int n = (k * 8 + lane) * V;
            if (r >= per || n >= N) continue;
            float v[V];
            Pack<DnT, V> out;
            decode<kType, V>(p[i][k], v);
#pragma unroll
            for (int j = 0; j < V; ++j) out.v[j] = from_float<DnT>(init ? v[j] * scale[i] : 0.f);
            store_pack<DnT, V>(dst + n, out);
        }
    }
}

template <bool kStore, typename DnT, int kType, int E, int V>
cudaError_t launch(const ssd_state_params &p, cudaStream_t stream) {
    const int64_t per = (int64_t)p.nheads * p.headdim, blocks = (per + kTile - 1) / kTile;
    if (p.num_states * blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(p.num_states * blocks));
    auto run = [&](auto kernel) { return enqueue(kernel, grid, kThreads, stream, p, (int)blocks); };
    if constexpr (kStore)
        return p.sr_seed ? run(store_kernel<DnT, kType, E, V, true>) : run(store_kernel<DnT, kType, E, V, false>);
    else
        return run(load_kernel<DnT, kType, E, V>);
}

template <bool kStore, typename DnT, int kType, int V>
cudaError_t launch_n(const ssd_state_params &p, cudaStream_t stream) {
    if (p.dstate <= 64) return launch<kStore, DnT, kType, 8, V>(p, stream);
    if (p.dstate <= 128) return launch<kStore, DnT, kType, 16, V>(p, stream);
    return launch<kStore, DnT, kType, 32, V>(p, stream);
}

// 16 bytes of the dense states a load where rows and bases allow it, then 4 values, then 1
template <bool kStore, typename DnT, int kType>
cudaError_t launch_vec(const ssd_state_params &p, cudaStream_t stream) {
    const int io = (int)sizeof(DnT);
    auto can = [&](int v) { return p.dstate % v == 0 && aligned_to(p.state_cache, v) && aligned_to(p.states, (size_t)v * io); };
    if constexpr (sizeof(DnT) == 2)
        if (p.dstate >= 64 && can(8)) return launch_n<kStore, DnT, kType, 8>(p, stream);
    return can(4) ? launch_n<kStore, DnT, kType, 4>(p, stream) : launch_n<kStore, DnT, kType, 1>(p, stream);
}

template <bool kStore>
cudaError_t launch_any(const ssd_state_params &p, cudaStream_t stream) {
    if (p.dense_dtype == SSD_F32)
        return p.state_dtype == SSD_E4M3 ? launch_vec<kStore, float, SSD_E4M3>(p, stream)
                                         : launch_vec<kStore, float, SSD_I8>(p, stream);
    return p.state_dtype == SSD_E4M3 ? launch_vec<kStore, __nv_bfloat16, SSD_E4M3>(p, stream)
                                     : launch_vec<kStore, __nv_bfloat16, SSD_I8>(p, stream);
}

}  // namespace

cudaError_t launch_state_store(const ssd_state_params &p, cudaStream_t stream) { return launch_any<true>(p, stream); }
cudaError_t launch_state_load(const ssd_state_params &p, cudaStream_t stream) { return launch_any<false>(p, stream); }

}  // namespace ssd
