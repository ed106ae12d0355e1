// Single-token step of a Mamba2 mixer: convolution, dt, state update, read-out
// and gate of one token per request, in one launch.
//
//   u = act(bias + sum_k w[:, W-1-k] xbc_{pos-k}),   u = (x, B, C)
//   h <- exp(dt' A) h + dt' x B^T,   y = (C h + D x) SiLU(z)
//
// The state is read once and written once and dwarfs the rest (N values for
// each x): the kernel is bound by HBM, for small batches by latency.
//
// A request's states are H P rows of N values; the rows of a group share B and
// C.  A CTA takes a run of one group's rows, whatever heads they belong to,
// sixteen or 32 at a time.  Eight or four lanes share a row, so that its sums and
// maxima take two or three shuffles, and a warp's rows are neighbours in memory.  A thread
// copies its own share of the next rows into shared memory asynchronously, a
// few steps ahead, and alone reads it back: no barriers, no registers for data
// in flight, and the first copies run while the convolution, which needs the
// same indices, loads its inputs.
//
// The convolution cache is a ring, so the row the call writes (pos mod rows)
// is none of those its other CTAs read, and they need no order among them.
// Every CTA convolves its group's B and C for itself (from L2).
//
// Where a rounding of the last place can show in what a program sees later,
// everything that leads to the stored state is rounded operation by operation,
// sums from the oldest tap on, so that a plain fp32 program stores the same
// bits: with every 8-bit cache (a code that tips moves the scale of its whole row
// if it is the row's largest), with a seeded fp16 one, and with fp32 activations
// and any cache below fp32 (a value that is rounded the other way is off by a
// step of its type, which fp32 outputs of later steps show).  Otherwise, with
// bf16 activations, products and sums are fused.
//
// Measured, 128 requests of 128 heads x 64 rows x 128 values: fp32 cache 164 us,
// 6.6 TB/s (98 % of the copy rate); bf16 86 us (94 %); e4m3 75 us to nearest and
// 112 us stochastically (57 and 38 %), bound by instructions: Philox 21 us of
// it, the roundings one by one 11.  One request, fp32: 3.3 us in a graph.
#pragma once

#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kStepThreads = 128;
constexpr int kStepMaxRows = 512;                  // of one CTA

// CTAs of an SM that the registers leave room for
template <int kType, int E>
constexpr int kStepCtas = E == 32 ? 4 : kType == SSD_E4M3 || kType == SSD_I8 ? 5 : 6;

struct StepPlan {
    int rows_g;        // rows of a group
    int rows;          // rows of a CTA, a multiple of 32
    int channels;
    int vec4;          // four channels and four rows make aligned vectors, and the width is 2, 3 or 4
    uint32_t p_mul;    // x / P = x p_mul >> p_shift for 0 <= x < 2^31
    int p_shift;
};

// floor(x / P) for all 0 <= x < 2^31: with 2^s >= P and m = ceil(2^(31+s) / P),
// m P - 2^(31+s) < 2^s, so x m / 2^(31+s) exceeds x / P by less than 1 / P.
inline void set_divisor(StepPlan &plan, int P) {
    int s = 0;
    while ((1LL << s) < P) ++s;
    plan.p_mul = (uint32_t)(((1ULL << (31 + s)) + P - 1) / P);
    plan.p_shift = 31 + s;
}

// acc + w x, and the activation of the sum with its bias: fused and approximated,
// or (plain) operation by operation
template <bool plain> __device__ __forceinline__ float tap(float acc, float w, float x) {
    return plain ? __fadd_rn(acc, __fmul_rn(w, x)) : fmaf(w, x, acc);
}
template <bool plain> __device__ __forceinline__ float convolved(float acc, float bias, int activation) {
    acc = __fadd_rn(acc, bias);
    if (!activation) return acc;
    return plain ? silu_stepwise(acc) : silu(acc);
}

// One channel's convolution at position pos.
template <typename IoT, bool plain>
__device__ __forceinline__ float conv_channel(const ssd_step_params &a, const IoT *xbc, const IoT *ring, int channels,
                                              int c, int pos, int row) {
    const IoT *w = static_cast<const IoT *>(a.weight) + (int64_t)c * a.width;
    float acc = 0.f;
#pragma unroll
    for (int k = SSD_CONV_MAX_WIDTH - 1; k > 0; --k) {
        if (k < a.width && k <= pos) {
            int r = row - k;
            if (r < 0) r += a.conv_rows;
            acc = tap<plain>(acc, to_float(w[a.width - 1 - k]), to_float(ring[(int64_t)r * channels + c]));
        }
    }
    acc = tap<plain>(acc, to_float(w[a.width - 1]), to_float(xbc[c]));
    return convolved<plain>(acc, a.bias ? to_float(static_cast<const IoT *>(a.bias)[c]) : 0.f, a.activation);
}

// Four neighbouring channels, all loads issued together.
template <typename IoT, bool plain, int kW>
__device__ __forceinline__ float4 conv_channels4(const ssd_step_params &a, const IoT *xbc, IoT *ring, int channels,
                                                 int c, int pos, int row, bool keep) {
    const Pack<IoT, 4 * kW> w = load_pack<IoT, 4 * kW>(static_cast<const IoT *>(a.weight) + (int64_t)c * kW);
    Pack<IoT, 4> in[kW], bias{};
    in[0] = load_pack<IoT, 4>(xbc + c);
#pragma unroll
    for (int k = 1; k < kW; ++k) {
        int r = row - k;
        if (r < 0) r += a.conv_rows;
        in[k] = Pack<IoT, 4>{};
        if (k <= pos) in[k] = load_pack<IoT, 4>(ring + (int64_t)r * channels + c);
    }
    if (a.bias) bias = load_pack<IoT, 4>(static_cast<const IoT *>(a.bias) + c);
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float acc = 0.f;
#pragma unroll
        for (int k = kW - 1; k >= 0; --k) acc = tap<plain>(acc, to_float(w.v[kW * j + kW - 1 - k]), to_float(in[k].v[j]));
        u[j] = convolved<plain>(acc, to_float(bias.v[j]), a.activation);
    }
    if (keep) store_pack<IoT, 4>(ring + (int64_t)row * channels + c, in[0]);
    return make_float4(u[0], u[1], u[2], u[3]);
}

// dt' and the decay exp(dt' A) of a head
template <typename IoT>
__device__ __forceinline__ float2 head_terms(const ssd_step_params &a, int b, int h) {
    float dt = to_float(static_cast<const IoT *>(a.dt)[(int64_t)b * a.dt_stride + h]);
    if (a.dt_bias) dt += a.dt_bias[h];
    if (a.dt_softplus) dt = softplus(dt);
    return make_float2(dt, expf(__fmul_rn(dt, a.A[h])));
}

// kType: storage of the state; L: lanes of a row; E: state values a lane holds
// of it (L E >= N); V: values of one copy; kDepth: row steps copied ahead; kSr:
// stochastic rounding; kF32Io: fp32 activations, else bf16 ones (an fp32 cache's
// kernel takes either).
template <int kType, int L, int E, int V, int kDepth, bool kSr, bool kF32Io>
__global__ void __launch_bounds__(kStepThreads, kStepCtas<kType, E>) step_kernel(const ssd_step_params a, const StepPlan plan) {
    using StT = typename Stored<kType>::T;
    constexpr int kChunks = E / V, kStepGroups = kStepThreads / L;     // rows worked on at a time
    constexpr bool k8bit = kType == SSD_E4M3 || kType == SSD_I8;
    constexpr bool stepwise = k8bit || kSr || (kF32Io && kType != SSD_F32);    // see above
    constexpr bool kAsync = V * sizeof(StT) >= 4;       // narrower shares are loaded when they are needed
    // of each row: D x, later y; dt' x; the decay
    __shared__ __align__(16) float s_b[L * E], s_c[L * E], s_y[kStepMaxRows], s_dx[kStepMaxRows], s_keep[kStepMaxRows];
    __shared__ __align__(16) float s_scale[k8bit ? kStepMaxRows : 4];       // of each row: the old scale, then the new one
    __shared__ __align__(16) uint32_t s_keys[kSr ? 20 : 1];
    constexpr bool kRowBytes = kSr && k8bit && V < 16;       // random bytes by rows, not by lanes
    __shared__ uint4 s_rand[kRowBytes ? kStepGroups * rand_blocks(L * E) : 1];
    __shared__ Pack<StT, V> s_raw[kAsync ? kDepth * kChunks * kStepThreads : 1];

    await_previous();
    const int N = a.dstate, P = a.headdim, H = a.nheads;
    const int b = blockIdx.x, g = blockIdx.y, run = blockIdx.z;
    const int tid = threadIdx.x, lane = tid % L, grp = tid / L;
    const int r0 = g * plan.rows_g + run * plan.rows;        // the CTA's rows of the request: r0 .. r0 + rows - 1
    const int rows = min(plan.rows, plan.rows_g - run * plan.rows);
    const bool bf16 = kType == SSD_F32 ? a.io_dtype == SSD_BF16 : !kF32Io;

    const int slot = a.slot_idx[(int64_t)b * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
    const int pos = a.pos[b];
    const int64_t y0 = (int64_t)b * H * P + r0;
    if (slot < 0 || slot >= a.num_slots || pos < 0) {
        if (slot == -1) {
            for (int i = tid; i < rows; i += kStepThreads) {
                if (bf16) static_cast<__nv_bfloat16 *>(a.out_y)[y0 + i] = __float2bfloat16_rn(0.f);
                else static_cast<float *>(a.out_y)[y0 + i] = 0.f;
            }
        } else if (tid == 0 && run == 0 && g == 0 && a.device_status) {
            atomicOr(a.device_status, pos < 0 ? SSD_DEV_BAD_POS : SSD_DEV_BAD_SLOT);
        }
        return;
    }

    // ---- the state's first copies ------------------------------------------
    const int64_t row0 = (int64_t)slot * H * P + r0;    // row of the cache
    StT *cache = static_cast<StT *>(a.state_cache) + row0 * N;
    // the next kStepGroups rows, to the stage's places; none at position 0
    const StT *ahead = cache + (int64_t)grp * N + lane * V;
    int ahead_rows = (pos > 0 ? rows : 0) - grp;        // how many from this thread's next on
    auto copy_rows = [&](int stage) {
        if constexpr (kAsync) {
            const bool live = ahead_rows > 0;
            const StT *src = live ? ahead : cache;
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
                copy_async<V * (int)sizeof(StT)>(&s_raw[(stage * kChunks + k) * kStepThreads + tid],
                                                 (k * L + lane) * V < N ? src + k * L * V : cache,
                                                 live && (k * L + lane) * V < N);
            commit_async();
            ahead += kStepGroups * N;
            ahead_rows -= kStepGroups;
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) copy_rows(d);

    // ---- convolution, and what each row takes from it and from its head -----
    const int channels = plan.channels;
    const int ring_row = pos % a.conv_rows;
    const int cb = H * P + g * N, cc = cb + a.ngroups * N;      // first channels of B and C
    auto convolve = [&](auto io) {
        using IoT = decltype(io);
        constexpr bool plain = stepwise || sizeof(IoT) == 4;
        const IoT *xbc = static_cast<const IoT *>(a.xbc) + (int64_t)b * a.xbc_stride;
        IoT *ring = static_cast<IoT *>(a.conv_cache) + (int64_t)slot * a.conv_rows * channels;
        auto head_of = [&](int row) { return (int)((uint64_t)(uint32_t)row * plan.p_mul >> plan.p_shift); };
        auto four = [&](int c, bool keep) {
            if (a.width == 4) return conv_channels4<IoT, plain, 4>(a, xbc, ring, channels, c, pos, ring_row, keep);
            if (a.width == 3) return conv_channels4<IoT, plain, 3>(a, xbc, ring, channels, c, pos, ring_row, keep);
            return conv_channels4<IoT, plain, 2>(a, xbc, ring, channels, c, pos, ring_row, keep);
        };
        if (plan.vec4) {
            for (int i = 4 * tid; i < 2 * N + rows; i += 4 * kStepThreads) {
                if (i < 2 * N) {
                    const int c = i < N ? cb + i : cc + i - N;
                    *reinterpret_cast<float4 *>(i < N ? s_b + i : s_c + i - N) =
                        four(c, run == 0);
                } else {
                    const int r = i - 2 * N, h = head_of(r0 + r);
                    float4 sc{};
                    if (k8bit) sc = *reinterpret_cast<const float4 *>(a.state_scale + row0 + r);
                    const float2 ht = head_terms<IoT>(a, b, h);
                    const float dh = a.D ? a.D[h] : 0.f;
                    const float4 x = four(r0 + r, true);
                    const float dt = ht.x, keep = pos > 0 ? ht.y : 0.f;
                    if (pos == 0) sc = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k8bit) *reinterpret_cast<float4 *>(s_scale + r) = sc;
                    *reinterpret_cast<float4 *>(s_dx + r) = make_float4(dt * x.x, dt * x.y, dt * x.z, dt * x.w);
                    *reinterpret_cast<float4 *>(s_y + r) = make_float4(dh * x.x, dh * x.y, dh * x.z, dh * x.w);
                    *reinterpret_cast<float4 *>(s_keep + r) = make_float4(keep, keep, keep, keep);
                }
            }
        } else {
            for (int i = tid; i < 2 * N + rows; i += kStepThreads) {
                const int c = i < N ? cb + i : i < 2 * N ? cc + i - N : r0 + i - 2 * N;
                const float u = conv_channel<IoT, plain>(a, xbc, ring, channels, c, pos, ring_row);
                if (i >= 2 * N || run == 0) ring[(int64_t)ring_row * channels + c] = xbc[c];
                if (i < 2 * N) {
                    *(i < N ? s_b + i : s_c + i - N) = u;
                } else {
                    const int r = i - 2 * N, h = head_of(r0 + r);
                    const float2 ht = head_terms<IoT>(a, b, h);
                    s_dx[r] = ht.x * u;
                    s_y[r] = a.D ? a.D[h] * u : 0.f;
                    if (k8bit) s_scale[r] = pos > 0 ? a.state_scale[row0 + r] : 0.f;
                    s_keep[r] = pos > 0 ? ht.y : 0.f;
                }
            }
        }
    };
    if (kSr && tid < 20) round_keys(*a.sr_seed, tid, s_keys);
    for (int i = N + tid; i < L * E; i += kStepThreads) s_b[i] = s_c[i] = 0.f;
    if constexpr (kType == SSD_F32 || !kF32Io)
        if (bf16) convolve(__nv_bfloat16{});
    if constexpr (kType == SSD_F32 || kF32Io)
        if (!bf16) convolve(float{});
    __syncthreads();

    // ---- update and read-out -----------------------------------------------
    float2 bv[E / 2], cv[E / 2];
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = k * V + j, n = (k * L + lane) * V + j;
            (e & 1 ? bv[e / 2].y : bv[e / 2].x) = s_b[n];
            (e & 1 ? cv[e / 2].y : cv[e / 2].x) = s_c[n];
        }
    int stage = 0;
    StT *dst = cache + (int64_t)grp * N + lane * V;
    uint64_t e0 = (uint64_t)(row0 + grp) * N + lane * V;        // flat index of the thread's first value
#pragma unroll 1
    for (int t = 0; t < rows; t += kStepGroups, dst += kStepGroups * N, e0 += kStepGroups * N) {
        const int r = t + grp;
        const bool live = r < rows;
        const float dx = s_dx[r], keep = s_keep[r];     // whatever they are past the last row
        const float2 dx2 = make_float2(dx, dx), keep2 = make_float2(keep, keep);
        float2 acc = make_float2(0.f, 0.f);
        float st[E];
        float big = 0.f;
        if constexpr (kAsync) wait_async<kDepth - 1>();
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const int n = (k * L + lane) * V;
            if (n >= N) continue;       // past the row: an infinite x must not meet a zero there
            Pack<StT, V> now{};
            if constexpr (kAsync) now = s_raw[(stage * kChunks + k) * kStepThreads + tid];
            else if (live && pos > 0) now = load_pack<StT, V>(dst + k * L * V);
            decode<kType, V>(now, st + k * V);
            if constexpr (stepwise && V == 1) {
                if (k8bit) st[k] = __fmul_rn(st[k], s_scale[r]);
                st[k] = __fadd_rn(__fmul_rn(keep, st[k]), __fmul_rn(dx, k & 1 ? bv[k / 2].y : bv[k / 2].x));
                acc.x = fmaf(k & 1 ? cv[k / 2].y : cv[k / 2].x, st[k], acc.x);
                if (k8bit) big = max_abs(big, st[k], st[k]);
            } else if constexpr (stepwise) {
                const float sc = k8bit ? s_scale[r] : 1.f;
#pragma unroll
                for (int e = k * V; e < (k + 1) * V; e += 2) {
                    float2 s = make_float2(st[e], st[e + 1]);
                    if (k8bit) s = mul2(s, make_float2(sc, sc));
                    const float2 old = mul2(keep2, s), add = mul2(dx2, bv[e / 2]);
                    s = make_float2(__fadd_rn(old.x, add.x), __fadd_rn(old.y, add.y));
                    acc = fma2(cv[e / 2], s, acc);
                    st[e] = s.x;
                    st[e + 1] = s.y;
                    if (k8bit) big = max_abs(big, s.x, s.y);
                }
            } else if constexpr (V == 1) {
                st[k] = fmaf(keep, st[k], dx * (k & 1 ? bv[k / 2].y : bv[k / 2].x));
                acc.x = fmaf(k & 1 ? cv[k / 2].y : cv[k / 2].x, st[k], acc.x);
            } else {
#pragma unroll
                for (int e = k * V; e < (k + 1) * V; e += 2) {
                    const float2 s = fma2(keep2, make_float2(st[e], st[e + 1]), mul2(dx2, bv[e / 2]));
                    acc = fma2(cv[e / 2], s, acc);
                    st[e] = s.x;
                    st[e + 1] = s.y;
                }
            }
        }
        // the values are in registers: their places take the rows kDepth steps on
        copy_rows(stage);
        stage = stage + 1 == kDepth ? 0 : stage + 1;
        const float sum = lanes_sum<L>(acc.x + acc.y);
        if (lane == 0 && live) s_y[r] += sum;
        float inv = 0.f, sc = 0.f;
        if constexpr (k8bit) {
            const float most = lanes_max<L>(big);
            row_scale(most, code_limit<kType>(), &inv, &sc);
            if (lane == 0 && live) s_scale[r] = sc;
        }
        uint4 *rand = s_rand + (kRowBytes ? grp * rand_blocks(L * E) : 0);
        if constexpr (kRowBytes) row_bytes<L>(rand, s_keys, e0 - lane * V, N, lane);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const int n = (k * L + lane) * V;
            if (!live || n >= N) continue;
            const float *v = st + k * V;
            const uint64_t e = e0 + k * L * V;
            Pack<StT, V> p;
            if constexpr (kType == SSD_F32) {
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = v[j];
            } else if constexpr (kType == SSD_BF16) {
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = __float2bfloat16_rn(v[j]);
            } else if constexpr (kType == SSD_F16) {
                if constexpr (kSr) {
                    uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if constexpr (V >= 4) {         // e is a multiple of 4
                            if (j % 4 == 0) w = sr_keyed(s_keys, (e + j) >> 2, 0u);
                            p.v[j] = sr_f16_fast(v[j], sr_word(w, j % 4));
                        } else {
                            w = sr_keyed(s_keys, (e + j) >> 2, 0u);
                            p.v[j] = sr_f16_fast(v[j], sr_word(w, (uint32_t)(e + j) & 3u));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) p.v[j] = __float2half_rn(v[j]);
                }
            } else {
                if constexpr (kSr) p = encode8_sr<kType, V>(v, inv, s_keys, e, reinterpret_cast<const uint8_t *>(rand) + ((e0 - lane * V) & 15) + n);
                else p = encode8<kType, V>(v, inv);
            }
            store_pack<StT, V>(dst + k * L * V, p);
        }
    }
    if constexpr (kAsync) wait_async<0>();
    __syncthreads();

    // ---- y ------------------------------------------------------------------
    for (int i = tid; i < rows; i += kStepThreads) {
        if (k8bit) a.state_scale[row0 + i] = s_scale[i];
        float y = s_y[i];
        if (bf16) {
            if (a.z) y *= silu(__bfloat162float(static_cast<const __nv_bfloat16 *>(a.z)[(int64_t)b * a.z_stride + r0 + i]));
            static_cast<__nv_bfloat16 *>(a.out_y)[y0 + i] = __float2bfloat16_rn(y);
        } else {
            if (a.z) y *= silu(static_cast<const float *>(a.z)[(int64_t)b * a.z_stride + r0 + i]);
            static_cast<float *>(a.out_y)[y0 + i] = y;
        }
    }
}

template <int kType, int L, int E, int V>
cudaError_t launch_step(const ssd_step_params &p, cudaStream_t stream) {
    constexpr int size = (int)sizeof(typename Stored<kType>::T);
    // steps in flight: 24 KB of a CTA's states (8 KB of 8-bit ones, whose CTAs
    // compute longer on them), at least two, at most six
    constexpr int kFit = (size == 1 ? 8192 : 24576) / (kStepThreads * E * size);
    constexpr int kDepth = kFit < 2 ? 2 : kFit > 6 ? 6 : kFit;
    StepPlan plan;
    const int rows_g = plan.rows_g = p.nheads / p.ngroups * p.headdim;
    plan.channels = p.nheads * p.headdim + 2 * p.ngroups * p.dstate;
    set_divisor(plan, p.headdim);
    // the run whose waves of CTAs take the least, a CTA's own start counted as 64
    // rows: long runs share the convolution of B and C, short ones fill the GPU
    constexpr int kMinRows = kStepThreads / L < 32 ? 32 : kStepThreads / L;
    const int64_t resident = 152 * kStepCtas<kType, E>;
    int64_t least = INT64_MAX;
    for (int rows = kMinRows; rows <= kStepMaxRows; rows += 32) {
        const int64_t ctas = (int64_t)((rows_g + rows - 1) / rows) * p.ngroups * p.batch;
        const int64_t cost = (ctas + resident - 1) / resident * (rows + 64);
        if (cost < least) {
            least = cost;
            plan.rows = rows;
        }
        if (rows >= rows_g) break;
    }
    const int runs = (rows_g + plan.rows - 1) / plan.rows;
    const int io = p.io_dtype == SSD_F32 ? 4 : 2, vec = 4 * io;
    plan.vec4 = p.width >= 2 && p.width <= 4 && p.dstate % 4 == 0 && p.headdim % 4 == 0 && p.xbc_stride % 4 == 0 &&
                aligned_to(p.xbc, vec) && aligned_to(p.conv_cache, vec) && aligned_to(p.bias, vec) &&
                aligned_to(p.weight, 16) && aligned_to(p.state_scale, 16);
    if (p.ngroups > 65535 || runs > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)p.batch, (unsigned)p.ngroups, (unsigned)runs);
    auto run = [&](auto kernel) { return enqueue(kernel, grid, kStepThreads, stream, p, plan); };
    const bool f32 = p.io_dtype == SSD_F32;
    if constexpr (kType == SSD_F32) return run(step_kernel<kType, L, E, V, kDepth, false, false>);
    if constexpr (kType != SSD_F32 && kType != SSD_BF16)
        if (p.sr_seed)
            return f32 ? run(step_kernel<kType, L, E, V, kDepth, true, true>)
                       : run(step_kernel<kType, L, E, V, kDepth, true, false>);
    if constexpr (kType != SSD_F32)
        return f32 ? run(step_kernel<kType, L, E, V, kDepth, false, true>)
                   : run(step_kernel<kType, L, E, V, kDepth, false, false>);
}

template <int kType, int L, int E>
cudaError_t launch_step_vec(const ssd_step_params &p, cudaStream_t stream) {
    constexpr int size = (int)sizeof(typename Stored<kType>::T);
    const int v = state_vector(p.dstate, size, p.state_cache, L);
    if constexpr (16 / size <= E) if (v == 16 / size) return launch_step<kType, L, E, 16 / size>(p, stream);
    if constexpr (4 <= E) if (v == 4) return launch_step<kType, L, E, 4>(p, stream);
    return launch_step<kType, L, E, 1>(p, stream);
}

// Eight lanes a row; four where a row of up to 64 narrow values would leave
// eight with less than a vector each.  (128 values a row, 128 requests, four lanes
// of 32 values instead: bf16 89 for 86 us, e4m3 68 for 64.)
template <int kType>
cudaError_t launch_step_type(const ssd_step_params &p, cudaStream_t stream) {
    if (p.dstate <= 16) return launch_step_vec<kType, 4, 4>(p, stream);
    if constexpr (kType == SSD_F32) {
        if (p.dstate <= 32) return launch_step_vec<kType, 8, 4>(p, stream);
        if (p.dstate <= 64) return launch_step_vec<kType, 8, 8>(p, stream);
    } else {
        if (p.dstate <= 32) return launch_step_vec<kType, 4, 8>(p, stream);
        if (p.dstate <= 64) return launch_step_vec<kType, 4, 16>(p, stream);
    }
    if (p.dstate <= 128) return launch_step_vec<kType, 8, 16>(p, stream);
    return launch_step_vec<kType, 8, 32>(p, stream);
}

}  // namespace
}  // namespace ssd
