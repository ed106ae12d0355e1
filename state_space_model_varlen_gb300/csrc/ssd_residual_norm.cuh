// Residual addition and RMS norm, with an output in 8 bits.  One translation unit
// for each type of x.
//
//   v = x + residual;  n = v / sqrt(mean(v^2) + eps) weight;  codes of n by groups
//
// Each value is read once and written once: bound by HBM.  Four to 32 lanes take a
// short row, a CTA a longer one; either holds the row in registers from the sum of
// squares to the stores, all its loads issued together.  The largest magnitude of a group
// of 1, 2, 4 .. 32 vectors comes from the lanes that hold it, of others from one entry
// a vector in shared memory.
//
// Measured: 16,384 rows of 2,560 bf16 columns with an fp32 residual 73 us, 6.87 TB/s (at
// the copy rate); 61,773 rows of 4,096 with a bf16 residual to e4m3 codes by groups of
// 128 289 us, 6.15 TB/s (91 %); one row of 4,096 2.3 us in a graph.  Read again for the norm
// and the codes instead of kept: 331 and 1,959 us.  Odd dense rows, whose vectors begin at
// the boundary before the row: 21,897 x 2,009 fp32 54 us (96 %; element by element 86),
// 30,000 x 2,001 bf16 with a bf16 residual 126 us (56 %: a weight at a time, and the ends;
// vectors of eight 141, weights put together from two vectors 147); even bf16 rows in
// pairs, 34,830 x 894 33 us (56 %).  Rows that registers do not hold, 4,000 x 20,000 fp32,
// element by element 473 us (40 %).  46,479 rows of 32 with codes 7 us, 21 with a warp a row.
#pragma once

#include <type_traits>

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

__device__ __forceinline__ void code_scale(const ssd_residual_norm_params &a, float m, float *inv, float *scale) {
    row_scale(m, a.code_dtype == SSD_E4M3 ? code_limit<SSD_E4M3>() : code_limit<SSD_I8>(), inv, scale);
}

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
        code_scale(a, m, &inv, &scale);
        if (lane == 0) row.scale[g] = scale;
        for (int i = lane; i < G; i += 32) {
            const int c = g * G + i;
            const float v = row.sum(c), n = row.normed(v, r, c);
            row.store(c, v, n);
            row.codes[c] = a.code_dtype == SSD_E4M3 ? encode1<SSD_E4M3>(n, inv) : encode1<SSD_I8>(n, inv);
        }
    }
}

// V consecutive values as pairs and back (V = 1: the first of a pair)
template <typename T, int V> __device__ __forceinline__ void unpack(const Pack<T, V> &p, float2 (&f)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        f[0] = make_float2(to_float(p.v[0]), 0.f);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) f[j] = pair_of<V>(p, j);
    }
}
template <typename T, int V> __device__ __forceinline__ Pack<T, V> packed(const float2 (&f)[(V + 1) / 2]) {
    Pack<T, V> p;
    if constexpr (V == 1) {
        p.v[0] = from_float<T>(f[0].x);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) set_pair<V>(p, j, f[j]);
    }
    return p;
}

constexpr int kRowThreads = 128;        // of a CTA that takes several rows
constexpr int kParts = 32;              // sums of a CTA's warps
constexpr size_t kMostShared = 48 * 1024 - kParts * sizeof(float);      // beside them, of a launch without an opt-in
template <int V> constexpr int kMost = V <= 2 ? 1024 : 512;     // of one that takes one row: what the registers allow

// V values from column c on, or those of them that the row has; and back
template <bool kShift, typename T, int V> __device__ __forceinline__ Pack<T, V> get(const T *row, int c, int columns) {
    if (!kShift || (c >= 0 && c + V <= columns)) return load_pack<T, V>(row + c);
    Pack<T, V> p{};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (c + j >= 0 && c + j < columns) p.v[j] = row[c + j];
    return p;
}
template <bool kShift, typename T, int V> __device__ __forceinline__ void put(T *row, int c, int columns, const Pack<T, V> &p) {
    if (!kShift || (c >= 0 && c + V <= columns)) {
        store_pack<T, V>(row + c, p);
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (c + j >= 0 && c + j < columns) row[c + j] = p.v[j];
}

// kLanes: lanes that take a row (4 to 32), or 0: the CTA does; C: vectors of a thread at most.
// kShift: rows that begin anywhere, all alike: `first` + row stride elements behind a
// boundary of V; the vectors begin at the boundary, and the weights come one by one.
template <typename IoT, typename ResT, int V, int kLanes, int C, bool kCodes, bool kShift = false>
__global__ void __launch_bounds__(kLanes ? kRowThreads : kMost<V>)
    residual_norm_kernel(const ssd_residual_norm_params a, int lanes, int first) {
    extern __shared__ float most[];     // largest magnitude of a vector, then inv of a group
    __shared__ float part[kParts];
    constexpr int kPairs = (V + 1) / 2;
    await_previous();
    constexpr bool kWarp = kLanes != 0;
    const int id = kWarp ? threadIdx.x % (kWarp ? kLanes : 1) : threadIdx.x, team = kWarp ? kLanes : blockDim.x;
    int64_t number = blockIdx.x;
    if (kWarp) number = number * (kRowThreads / (kWarp ? kLanes : 1)) + threadIdx.x / (kWarp ? kLanes : 1);
    const bool live = !kWarp || number < a.rows;        // behind the last row: lanes that only take part in the sums
    if (!live) number = a.rows - 1;
    const int columns = live ? a.columns : 0;
    const Row<IoT, ResT> row(a, number);
    const int shift = kShift ? (int)((first + number * a.x_stride) % V) : 0;
    auto column = [&](int k) { return (k * team + id) * V - shift; };
    Pack<IoT, V> x[C], w[C];
    Pack<ResT, V> res[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int c = column(k);
        x[k] = w[k] = Pack<IoT, V>{};
        res[k] = Pack<ResT, V>{};
        if (c < columns) {
            x[k] = get<kShift, IoT, V>(row.x, c, columns);
            if (row.res) res[k] = get<kShift, ResT, V>(row.res, c, columns);
        }
    }
    // weights ahead of the sum too, unless they come one by one into too many registers
    auto weights = [&](int k) {
        const int c = column(k);
        if (!row.w || c >= columns) return;
        if constexpr (kShift) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j >= 0 && c + j < columns) w[k].v[j] = row.w[c + j];
        } else {
            w[k] = load_pack<IoT, V>(row.w + c);
        }
    };
    constexpr bool kEarly = V > 1 && !(kShift && V == 8);
    if constexpr (kEarly)
#pragma unroll
        for (int k = 0; k < C; ++k) weights(k);
    float2 v[C][kPairs], two = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        float2 r[kPairs];
        unpack<IoT, V>(x[k], v[k]);
        unpack<ResT, V>(res[k], r);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            if (row.res) v[k][j] = add2(v[k][j], r[j]);
            two = fma2(v[k][j], v[k][j], two);
        }
    }
    if (row.res_out)
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (column(k) < columns) put<kShift, ResT, V>(row.res_out, column(k), columns, packed<ResT, V>(v[k]));
    const float sum = kWarp ? lanes_sum<kWarp ? kLanes : 32>(two.x + two.y) : cta_sum(two.x + two.y, part);
    const float r = 1.f / sqrtf(sum / (float)a.columns + a.eps);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int c = column(k);
        if constexpr (!kEarly) weights(k);
        float2 f[kPairs];
        unpack<IoT, V>(w[k], f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            v[k][j] = mul2(v[k][j], make_float2(r, r));
            if (row.w) v[k][j] = mul2(v[k][j], f[j]);
        }
        if (row.out && c < columns) put<kShift, IoT, V>(row.out, c, columns, packed<IoT, V>(v[k]));
    }
    if constexpr (kCodes) {
        const int G = a.scale_group, per = G / V;       // vectors of a group
        float m[C];
#pragma unroll
        for (int k = 0; k < C; ++k) {
            m[k] = 0.f;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) m[k] = max_abs(m[k], v[k][j].x, v[k][j].y);
        }
        float inv[C];
        if (lanes > 0) {                // lanes that share a group, a power of two
            for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    const float u = __shfl_xor_sync(0xffffffffu, m[k], o);
                    m[k] = max_abs(m[k], u, u);
                }
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const int at = k * team + id;
                float scale;
                code_scale(a, m[k], &inv[k], &scale);
                if ((id & (lanes - 1)) == 0 && at * V < columns) row.scale[at / lanes] = scale;
            }
        } else {
            float *const mine = most + (kWarp ? (threadIdx.x >> 5) * (a.columns / V + a.columns / G) : 0);
            float *const invs = mine + a.columns / V;
            auto sync = [] {
                if constexpr (kWarp) __syncwarp();
                else __syncthreads();
            };
#pragma unroll
            for (int k = 0; k < C; ++k)
                if ((k * team + id) * V < columns) mine[k * team + id] = m[k];
            sync();
            const int lane = threadIdx.x & 31;
            for (int g = kWarp ? 0 : threadIdx.x >> 5; g < columns / G; g += kWarp ? 1 : team >> 5) {
                float u = 0.f;
                for (int i = lane; i < per; i += 32) u = max_abs(u, mine[g * per + i], mine[g * per + i]);
                u = lanes_max<32>(u);
                float scale, i;
                code_scale(a, u, &i, &scale);
                if (lane == 0) {
                    row.scale[g] = scale;
                    invs[g] = i;
                }
            }
            sync();
#pragma unroll
            for (int k = 0; k < C; ++k) inv[k] = (k * team + id) * V < columns ? invs[(k * team + id) / per] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int c = (k * team + id) * V;
            if (c >= columns) continue;
            float f[2 * kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                f[2 * j] = v[k][j].x;
                f[2 * j + 1] = v[k][j].y;
            }
            store_pack<uint8_t, V>(row.codes + c, a.code_dtype == SSD_E4M3 ? encode8<SSD_E4M3, V>(f, inv[k])
                                                                          : encode8<SSD_I8, V>(f, inv[k]));
        }
    }
}

template <typename IoT, typename ResT, int V, bool kCodes, bool kShift = false>
cudaError_t launch_row(const ssd_residual_norm_params &p, cudaStream_t stream, bool *taken, int first = 0) {
    const int vectors = kShift ? (p.columns + V - 2) / V + 1 : p.columns / V, per = kCodes ? p.scale_group / V : 1;
    const bool shuffled = per <= 32 && (per & (per - 1)) == 0;
    const int lanes = kCodes && shuffled ? per : 0;
    const size_t entries = kCodes && !shuffled ? (size_t)vectors + p.columns / p.scale_group : 0;
    auto go = [&](auto kernel, int64_t ctas, int threads, size_t rows) {
        if (ctas > 0x7fffffffLL || rows * entries * 4 > kMostShared) return cudaErrorInvalidConfiguration;
        *taken = true;
        return enqueue_shared(kernel, dim3((unsigned)ctas), threads, rows * entries * 4, stream, p, lanes, first);
    };
    constexpr int kShort = V == 1 ? 4 : 2;
    auto several = [&](auto kernel, int of_a_row) {     // rows of a CTA
        const int rows = kRowThreads / of_a_row;
        return go(kernel, (p.rows + rows - 1) / rows, kRowThreads, rows);
    };
    if constexpr (V >= 4 && !kShift)
        if (shuffled) {
            if (vectors <= 4) return several(residual_norm_kernel<IoT, ResT, V, 4, 1, kCodes>, 4);
            if (vectors <= 8) return several(residual_norm_kernel<IoT, ResT, V, 8, 1, kCodes>, 8);
            if (vectors <= 16) return several(residual_norm_kernel<IoT, ResT, V, 16, 1, kCodes>, 16);
        }
    if (vectors <= 32 * kShort) return several(residual_norm_kernel<IoT, ResT, V, 32, kShort, kCodes, kShift>, 32);
    auto whole = [&](auto kernel, int chunks) {
        return go(kernel, p.rows, 32 * ((vectors + 32 * chunks - 1) / (32 * chunks)), 1);
    };
    if constexpr (V == 1) {
        if (vectors <= kMost<V> * 10) return whole(residual_norm_kernel<IoT, ResT, V, 0, 10, kCodes>, 10);
    } else {
        if (vectors <= kMost<V> * 4) return whole(residual_norm_kernel<IoT, ResT, V, 0, 4, kCodes, kShift>, 4);
        if (vectors <= kMost<V> * 8) return whole(residual_norm_kernel<IoT, ResT, V, 0, 8, kCodes, kShift>, 8);
    }
    return cudaErrorInvalidConfiguration;
}

template <typename IoT, typename ResT> cudaError_t launch_norm(const ssd_residual_norm_params &p, cudaStream_t stream) {
    auto can = [&](int v) {
        const size_t io = v * sizeof(IoT) > 16 ? 16 : v * sizeof(IoT), res = v * sizeof(ResT) > 16 ? 16 : v * sizeof(ResT);
        return p.columns % v == 0 && p.x_stride % v == 0 && aligned_to(p.x, io) && aligned_to(p.weight, io) &&
               (!p.residual || (p.residual_stride % v == 0 && aligned_to(p.residual, res))) &&
               (!p.residual_out || (p.residual_out_stride % v == 0 && aligned_to(p.residual_out, res))) &&
               (!p.out || (p.out_stride % v == 0 && aligned_to(p.out, io))) &&
               (!p.out_codes || (p.scale_group % v == 0 && p.codes_stride % v == 0 && aligned_to(p.out_codes, v)));
    };
    bool taken = false;
    cudaError_t e = cudaErrorInvalidConfiguration;
    // rows that all begin alike, if not at a boundary: in vectors from the boundary on
    auto beside = [&](auto width) {
        constexpr int V = decltype(width)::value;
        const int first = (int)(reinterpret_cast<uintptr_t>(p.x) / sizeof(IoT) % V);
        auto alike = [&](const void *q, int64_t stride, size_t size) {
            return !q || ((int)(reinterpret_cast<uintptr_t>(q) / size % V) == first && (stride - p.x_stride) % V == 0);
        };
        if (p.out_codes || p.x_stride >= (1LL << 40) || !alike(p.residual, p.residual_stride, sizeof(ResT)) ||
            !alike(p.residual_out, p.residual_out_stride, sizeof(ResT)) || !alike(p.out, p.out_stride, sizeof(IoT)))
            return cudaErrorInvalidConfiguration;
        return launch_row<IoT, ResT, V, false, true>(p, stream, &taken, first);
    };
    auto row = [&](auto width) {
        constexpr int V = decltype(width)::value;
        return p.out_codes ? launch_row<IoT, ResT, V, true>(p, stream, &taken) : launch_row<IoT, ResT, V, false>(p, stream, &taken);
    };
    using std::integral_constant;
    if (sizeof(IoT) == 2 && can(8)) e = row(integral_constant<int, sizeof(IoT) == 2 ? 8 : 4>());
    else if (can(4)) e = row(integral_constant<int, 4>());
    else if (sizeof(IoT) == 2 && can(2)) e = row(integral_constant<int, sizeof(IoT) == 2 ? 2 : 1>());
    if (!taken && !can(4)) {
        if (sizeof(IoT) == 2 && p.columns > 8192) e = beside(integral_constant<int, sizeof(IoT) == 2 ? 8 : 4>());
        if (!taken) e = beside(integral_constant<int, 4>());
        if (!taken) e = row(integral_constant<int, 1>());
    }
    if (taken) return e;
    if (p.rows > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int threads = p.columns >= 1024 ? 1024 : (p.columns + 31) / 32 * 32;
    return enqueue(residual_norm_any_kernel<IoT, ResT>, dim3((unsigned)p.rows), threads, stream, p);
}

}  // namespace
}  // namespace ssd
