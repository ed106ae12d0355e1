// Gated RMS norm over groups of columns.
//
//   out = rms(y SiLU(z)) w   or   rms(y) w SiLU(z)
//
// Each value is read once and written once: bound by HBM.  Four to 32 lanes
// take a short group of one row, a CTA a longer one; either holds the group in
// registers between the sum of squares and the scaling, all its loads issued
// together.  Groups past what a CTA holds are read twice (from L2 the second
// time).
//
// Measured: 16,384 rows of 5,120 bf16 columns, one group each, 81 us, 6.2 TB/s
// (91 % of the copy rate); 1,048,576 groups of 64 72 us (82 %); an odd number of
// columns, loaded one by one, 189 us (39 %).  8,192 columns of one row 1.9 us in a graph.
#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kItemThreads = 128;           // of a CTA that takes several groups
// the most threads of a CTA that takes one group: what the registers allow
template <int V> constexpr int kThreads = V == 1 ? 1024 : 512;

// one group of one row
template <typename IoT> struct Item {
    const IoT *y, *z, *w;
    IoT *out;
    __device__ Item(const ssd_gated_norm_params &a, int64_t item, int groups) {
        const int64_t row = item / groups;
        const int c0 = (int)(item % groups) * a.group_size;
        y = static_cast<const IoT *>(a.y) + row * a.y_stride + c0;
        z = a.z ? static_cast<const IoT *>(a.z) + row * a.z_stride + c0 : nullptr;
        w = a.weight ? static_cast<const IoT *>(a.weight) + c0 : nullptr;
        out = static_cast<IoT *>(a.out) + row * a.out_stride + c0;
    }
};

// What is normed of a vector: y, or y SiLU(z).  (V = 1: the first of a pair.)
template <typename IoT, int V>
__device__ __forceinline__ void normed(const Pack<IoT, V> &y, const Pack<IoT, V> &z, bool gated, float2 (&v)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        v[0].x = to_float(y.v[0]);
        if (gated) v[0].x *= silu(to_float(z.v[0]));
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            v[j] = pair_of<V>(y, j);
            if (gated) v[j] = mul2(v[j], silu2(pair_of<V>(z, j)));
        }
    }
}
template <int V> __device__ __forceinline__ void add_squares(float2 &sum, const float2 (&v)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        sum.x = fmaf(v[0].x, v[0].x, sum.x);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) sum = fma2(v[j], v[j], sum);
    }
}
// v r w, times SiLU(z) where the gate comes after the norm
template <typename IoT, int V>
__device__ __forceinline__ Pack<IoT, V> scaled(const float2 (&v)[(V + 1) / 2], float r, const Pack<IoT, V> &w, bool weighted,
                                               const Pack<IoT, V> &z, bool gated) {
    Pack<IoT, V> o;
    if constexpr (V == 1) {
        float f = v[0].x * r;
        if (weighted) f *= to_float(w.v[0]);
        if (gated) f *= silu(to_float(z.v[0]));
        o.v[0] = from_float<IoT>(f);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            float2 f = mul2(v[j], make_float2(r, r));
            if (weighted) f = mul2(f, pair_of<V>(w, j));
            if (gated) f = mul2(f, silu2(pair_of<V>(z, j)));
            set_pair<V>(o, j, f);
        }
    }
    return o;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// over the CTA, whose warps leave their sums in part
__device__ __forceinline__ float cta_sum(float v, float *part) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < blockDim.x / 32 ? part[threadIdx.x & 31] : 0.f;
    return warp_sum(v);
}

// kLanes: lanes of an item, or 0: the CTA takes one; C: vectors of a thread at most.
template <typename IoT, int V, int kLanes, int C>
__global__ void __launch_bounds__(kLanes ? kItemThreads : kThreads<V>)
    gated_norm_kernel(const ssd_gated_norm_params a, int groups, int64_t items) {
    __shared__ float part[32];
    await_previous();
    constexpr int L = kLanes ? kLanes : 32;
    const int64_t id = kLanes ? ((int64_t)blockIdx.x * kItemThreads + threadIdx.x) / L : blockIdx.x;
    const bool live = id < items;               // past the last item: lanes that only take part in the sums
    const Item<IoT> it(a, live ? id : 0, groups);
    const int size = live ? a.group_size : 0;
    const int at = (kLanes ? threadIdx.x % L : threadIdx.x) * V, step = (kLanes ? L : blockDim.x) * V;
    const bool after = it.z && a.norm_before_gate, before = it.z && !a.norm_before_gate;
    Pack<IoT, V> y[C], z[C], w[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int c = at + k * step;
        y[k] = z[k] = w[k] = Pack<IoT, V>{};
        if (c < size) {
            y[k] = load_pack<IoT, V>(it.y + c);
            if (it.z) z[k] = load_pack<IoT, V>(it.z + c);
        }
    }
    // weights ahead of the sum too, unless they would take single elements a register each
    if constexpr (V > 1)
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (it.w && at + k * step < size) w[k] = load_pack<IoT, V>(it.w + at + k * step);
    float2 v[C][(V + 1) / 2], two = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        normed<IoT, V>(y[k], z[k], before, v[k]);
        add_squares<V>(two, v[k]);
    }
    const float sum = kLanes ? lanes_sum<L>(two.x + two.y) : cta_sum(two.x + two.y, part);
    const float r = 1.f / sqrtf(sum / (float)a.group_size + a.eps);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int c = at + k * step;
        if (c >= size) continue;
        if (V == 1 && it.w) w[k] = load_pack<IoT, V>(it.w + c);
        store_pack<IoT, V>(it.out + c, scaled<IoT, V>(v[k], r, w[k], it.w != nullptr, z[k], after));
    }
}

template <typename IoT, int V>
__global__ void __launch_bounds__(1024) gated_norm_long_kernel(const ssd_gated_norm_params a, int groups) {
    __shared__ float part[32];
    await_previous();
    const Item<IoT> it(a, blockIdx.x, groups);
    const bool after = it.z && a.norm_before_gate, before = it.z && !a.norm_before_gate;
    float2 two = make_float2(0.f, 0.f);
    float r = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 4
        for (int c = threadIdx.x * V; c < a.group_size; c += blockDim.x * V) {
            Pack<IoT, V> y = load_pack<IoT, V>(it.y + c), z{}, w{};
            if (it.z) z = load_pack<IoT, V>(it.z + c);
            float2 v[(V + 1) / 2];
            normed<IoT, V>(y, z, before, v);
            if (pass) {
                if (it.w) w = load_pack<IoT, V>(it.w + c);
                store_pack<IoT, V>(it.out + c, scaled<IoT, V>(v, r, w, it.w != nullptr, z, after));
            } else {
                add_squares<V>(two, v);
            }
        }
        if (!pass) r = 1.f / sqrtf(cta_sum(two.x + two.y, part) / (float)a.group_size + a.eps);
    }
}

template <typename IoT, int V>
cudaError_t launch(const ssd_gated_norm_params &p, cudaStream_t stream) {
    const int groups = p.columns / p.group_size;
    const int64_t items = p.rows * groups;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int vectors = (p.group_size + V - 1) / V;
    auto shared = [&](auto kernel, int lanes) {
        const int64_t per = kItemThreads / lanes;
        return enqueue(kernel, dim3((unsigned)((items + per - 1) / per)), kItemThreads, stream, p, groups, items);
    };
    if (vectors <= 4) return shared(gated_norm_kernel<IoT, V, 4, 1>, 4);
    if (vectors <= 8) return shared(gated_norm_kernel<IoT, V, 8, 1>, 8);
    if (vectors <= 16) return shared(gated_norm_kernel<IoT, V, 16, 1>, 16);
    if (vectors <= 32) return shared(gated_norm_kernel<IoT, V, 32, 1>, 32);
    if (vectors <= 128) return shared(gated_norm_kernel<IoT, V, 32, 4>, 32);
    auto whole = [&](auto kernel, int chunks) {
        return enqueue(kernel, dim3((unsigned)items), 32 * ((vectors + 32 * chunks - 1) / (32 * chunks)), stream, p, groups,
                       items);
    };
    if constexpr (V == 1) {
        if (vectors <= kThreads<V> * 10) return whole(gated_norm_kernel<IoT, V, 0, 10>, 10);
    } else {
        if (vectors <= kThreads<V> * 4) return whole(gated_norm_kernel<IoT, V, 0, 4>, 4);
        if (vectors <= kThreads<V> * 8) return whole(gated_norm_kernel<IoT, V, 0, 8>, 8);
    }
    return enqueue(gated_norm_long_kernel<IoT, V>, dim3((unsigned)items), 1024, stream, p, groups);
}

}  // namespace

cudaError_t launch_gated_norm(const ssd_gated_norm_params &p, cudaStream_t stream) {
    const int io = p.io_dtype == SSD_F32 ? 4 : 2;
    auto can = [&](int v) {
        const size_t bytes = (size_t)v * io;
        return p.group_size % v == 0 && p.y_stride % v == 0 && p.out_stride % v == 0 && p.z_stride % v == 0 &&
               aligned_to(p.y, bytes) && aligned_to(p.z, bytes) && aligned_to(p.out, bytes) && aligned_to(p.weight, bytes);
    };
    if (p.io_dtype == SSD_F32) return can(4) ? launch<float, 4>(p, stream) : launch<float, 1>(p, stream);
    return can(8)   ? launch<__nv_bfloat16, 8>(p, stream)
           : can(4) ? launch<__nv_bfloat16, 4>(p, stream)
                    : launch<__nv_bfloat16, 1>(p, stream);
}

}  // namespace ssd
