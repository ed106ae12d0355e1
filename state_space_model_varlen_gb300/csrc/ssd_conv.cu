// Short causal convolution of packed prompts, split into the scan's inputs.
//
//   u_t[c] = act(bias[c] + sum_{k < W} w[c, W-1-k] xbc_{t-k}[c])
//
// Each value is read once and written once: the kernel is bound by HBM.  A CTA
// owns a tile of tokens and of channels; a thread owns V neighbouring channels
// and walks the tile's tokens in groups of eight with the last W - 1 inputs in
// registers.  It copies its own share of the inputs into shared memory
// asynchronously, a few groups ahead, and alone reads it back.  A tile reads
// W - 1 tokens more than it writes.
//
// Sequence boundaries are worked out once per CTA, while the first group's
// inputs are on their way: every thread looks at some of the sequences and
// marks the tile's tokens in shared memory.  A group whose tokens all have
// their W - 1 predecessors in this call slides the window; any other loads
// every tap of every token from where it lies, four tokens at a time.
//
// The convolution cache is updated in place by other CTAs than those that
// read it, unless one thread does both: the CTA whose tile holds a sequence's
// first token, which reads the ring, also writes the sequence's last inputs to
// it, afterwards, also where those lie in later tiles.
#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxTile = 64;       // tokens of a tile
constexpr int kGroup = 8;          // tokens whose inputs are loaded together
constexpr int kSlow = 2;           // tokens of a group at a boundary taken together

struct Token {
    int local;      // token of its sequence, -1: no valid sequence
    int row;        // its row of the ring
    int slot;       // -1: no cache
    int past;       // min(position, W - 1)
};
constexpr int kSlides = 1, kKeeps = 2;      // of a group: every token has its window here; some go to the ring

// dt of the tile's tokens widened to fp32
template <typename IoT>
__device__ __forceinline__ void widen_dt(const ssd_conv_params &a, int64_t t0, int nt) {
    const IoT *dt = static_cast<const IoT *>(a.dt);
    for (int h = threadIdx.x; h < a.nheads; h += kThreads) {
        for (int i = 0; i < nt; i += kGroup) {
            float v[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (i + j < nt) v[j] = to_float(dt[(t0 + i + j) * a.dt_stride + h]);
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (i + j < nt) a.out_dt[(t0 + i + j) * a.nheads + h] = v[j];
        }
    }
}

// A thread's channels as pairs of floats (V = 1: the first of one), acc += w x
// over them, and the finished values.
template <typename IoT, int V>
__device__ __forceinline__ void widen(const Pack<IoT, V> &x, float2 (&f)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        f[0].x = to_float(x.v[0]);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) f[j] = pair_of<V>(x, j);
    }
}
template <int V>
__device__ __forceinline__ void accumulate(float2 (&acc)[(V + 1) / 2], const float2 (&w)[(V + 1) / 2],
                                           const float2 (&x)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        acc[0].x = fmaf(w[0].x, x[0].x, acc[0].x);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) acc[j] = fma2(w[j], x[j], acc[j]);
    }
}
template <typename IoT, int V>
__device__ __forceinline__ Pack<IoT, V> finished(const float2 (&acc)[(V + 1) / 2], int activation) {
    Pack<IoT, V> u;
    if constexpr (V == 1) {
        u.v[0] = from_float<IoT>(activation ? silu(acc[0].x) : acc[0].x);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) set_pair<V>(u, j, activation ? silu2(acc[j]) : acc[j]);
    }
    return u;
}

// CTAs of an SM that the registers should leave room for
template <typename IoT, int V, int kW>
constexpr int kMinCtas = kW == 0 ? 2 : V * sizeof(IoT) > 8 ? 4 : 6;

// kW: the width, or 0 for one that only a.width tells (then no group slides).
template <typename IoT, int V, int kW>
__global__ void __launch_bounds__(kThreads, kMinCtas<IoT, V, kW>) conv_kernel(const ssd_conv_params a, int tile, int dt_column) {
    __shared__ int seq_of[kMaxTile];
    __shared__ Token token[kMaxTile];
    __shared__ uint8_t keep[kMaxTile];             // the token goes to the ring here
    __shared__ int group[kMaxTile / kGroup];
    __shared__ int tail_seq;
    constexpr int kM = kW ? kW : SSD_CONV_MAX_WIDTH;
    constexpr int kPast = kW > 1 ? kW - 1 : 1;      // inputs a sliding window keeps
    constexpr int kPairs = (V + 1) / 2;
    // groups copied ahead: 24 KB of a CTA's inputs; two-byte shares are loaded one group ahead instead
    constexpr int kBytes = V * (int)sizeof(IoT);
    constexpr bool kAsync = kBytes >= 4 && kW > 1;
    constexpr int kDepth = kBytes >= 16 ? 2 : kBytes == 8 ? 3 : 4;
    __shared__ Pack<IoT, V> s_x[kAsync ? kDepth * kGroup * kThreads : 1];
    const int W = kW ? kW : a.width;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)min((int64_t)tile, a.total_tokens - t0);
    const int ct = (int)blockIdx.y - dt_column;
    if (ct < 0) {
        widen_dt<IoT>(a, t0, nt);
        return;
    }
    const bool reporter = ct == 0 && a.device_status != nullptr;

    // ---- the first group's inputs and the window before it -----------------
    const int c = (ct * kThreads + threadIdx.x) * V;
    const bool mine = c < a.channels;
    const IoT *x = static_cast<const IoT *>(a.xbc) + t0 * a.xbc_stride + c;    // of the tile's first token
    Pack<IoT, V> next[kGroup], prev[kPast];
    auto load_group = [&](int i0, int stage) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            const bool live = mine && i0 + j < nt;
            if constexpr (kAsync)
                copy_async<kBytes>(&s_x[(stage * kGroup + j) * kThreads + threadIdx.x],
                                   live ? x + (i0 + j) * a.xbc_stride : static_cast<const IoT *>(a.xbc), live);
            else if (live)
                next[j] = load_pack<IoT, V>(x + (i0 + j) * a.xbc_stride);
        }
        if constexpr (kAsync) commit_async();
    };
    if constexpr (kW > 1) {
#pragma unroll
        for (int d = 0; d < (kAsync ? kDepth : 1); ++d) load_group(d * kGroup, d);
#pragma unroll
        for (int m = 1; m < kW; ++m) {
            prev[m - 1] = Pack<IoT, V>{};
            if (mine && t0 >= m) prev[m - 1] = load_pack<IoT, V>(x - m * a.xbc_stride);
        }
    }

    // ---- the tile's tokens -------------------------------------------------
    if (threadIdx.x < kMaxTile) seq_of[threadIdx.x] = -1;
    if (threadIdx.x < kMaxTile / kGroup) group[threadIdx.x] = kW > 1 ? kSlides : 0;
    if (threadIdx.x == 0) tail_seq = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < a.num_seqs; s += kThreads) {
        const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
        if (b < 0 || e < b || e > a.total_tokens) {
            if (t0 == 0 && reporter) atomicOr(a.device_status, SSD_DEV_BAD_SEQLENS);
            continue;
        }
        const int64_t lo = max(b, t0), hi = min(e, t0 + nt);
        for (int64_t t = lo; t < hi; ++t) seq_of[t - t0] = s;
    }
    __syncthreads();
    if (threadIdx.x < kMaxTile) {
        const int s = (int)threadIdx.x < nt ? seq_of[threadIdx.x] : -1;
        Token k = {-1, 0, -1, 0};
        bool kept = false;
        if (s >= 0) {
            const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
            const int64_t local = t0 + threadIdx.x - b;
            const int start = a.start_pos ? a.start_pos[s] : 0;
            int slot = -1;
            bool ok = true;
            if (a.conv_cache != nullptr) {
                slot = a.slot_idx[s * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
                ok = slot >= 0 && slot < a.num_slots;
                if (!ok && local == 0 && reporter) atomicOr(a.device_status, SSD_DEV_BAD_SLOT);
            }
            if (start < 0) {
                ok = false;
                if (local == 0 && reporter) atomicOr(a.device_status, SSD_DEV_BAD_POS);
            }
            if (ok) {
                const int64_t pos = start + local;
                const bool begins_here = b >= t0;
                k.local = (int)min(local, (int64_t)0x7fffffff);
                k.slot = slot;
                k.row = slot >= 0 ? (int)(pos % a.conv_rows) : 0;
                k.past = (int)min(pos, (int64_t)(W - 1));
                kept = slot >= 0 && begins_here && t0 + threadIdx.x >= e - (W - 1);
                // the tile's last sequence goes on after it: its end is kept below
                if (slot >= 0 && begins_here && (int)threadIdx.x == nt - 1 && e > t0 + nt) tail_seq = s;
            }
        }
        token[threadIdx.x] = k;
        keep[threadIdx.x] = kept;
        if (k.local < W - 1) atomicAnd(&group[threadIdx.x / kGroup], ~kSlides);
        if (kept) atomicOr(&group[threadIdx.x / kGroup], kKeeps);
    }
    __syncthreads();
    if (!mine) {
        if constexpr (kAsync) wait_async<0>();
        return;
    }

    IoT *ring = static_cast<IoT *>(a.conv_cache) + c;
    // where this thread's channels go
    IoT *out;
    int64_t ostride;
    if (c < a.split0) {
        out = static_cast<IoT *>(a.out0) + c;
        ostride = a.split0;
    } else if (c < a.split0 + a.split1) {
        out = static_cast<IoT *>(a.out1) + (c - a.split0);
        ostride = a.split1;
    } else {
        out = static_cast<IoT *>(a.out2) + (c - a.split0 - a.split1);
        ostride = a.channels - a.split0 - a.split1;
    }
    out += t0 * ostride;

    float2 w[kM][kPairs], bias[kPairs];        // w[k]: the tap of the token k before
    if constexpr (kW > 0 && V > 1) {
        const Pack<IoT, V * kM> pw = load_pack<IoT, V * kM>(static_cast<const IoT *>(a.weight) + (int64_t)c * kM);
        Pack<IoT, V> pb{};
        if (a.bias) pb = load_pack<IoT, V>(static_cast<const IoT *>(a.bias) + c);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            bias[j] = pair_of<V>(pb, j);
#pragma unroll
            for (int k = 0; k < kM; ++k)
                w[k][j] = make_float2(to_float(pw.v[2 * j * kM + kM - 1 - k]), to_float(pw.v[(2 * j + 1) * kM + kM - 1 - k]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float bj = a.bias ? to_float(static_cast<const IoT *>(a.bias)[c + j]) : 0.f;
            (j & 1 ? bias[j / 2].y : bias[j / 2].x) = bj;
#pragma unroll
            for (int k = 0; k < kM; ++k) {
                const float wk =
                    k < W ? to_float(static_cast<const IoT *>(a.weight)[(int64_t)(c + j) * W + (W - 1 - k)]) : 0.f;
                (j & 1 ? w[k][j / 2].y : w[k][j / 2].x) = wk;
            }
        }
    }

    float2 win[kPast][kPairs];          // win[m]: the input m + 1 tokens before
#pragma unroll
    for (int m = 0; m < kPast; ++m) widen<IoT, V>(prev[m], win[m]);
    int stage = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < nt; i0 += kGroup) {
        const int what = group[i0 / kGroup];
        if constexpr (kW > 1) {
            Pack<IoT, V> now[kGroup];
            if constexpr (kAsync) wait_async<kDepth - 1>();
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                now[i] = kAsync ? s_x[(stage * kGroup + i) * kThreads + threadIdx.x] : next[i];
            if constexpr (!kAsync) load_group(i0 + kGroup, 0);
            if (what & kSlides) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    float2 acc[kPairs], f[kPairs];
                    widen<IoT, V>(now[i], f);
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) acc[j] = bias[j];
                    accumulate<V>(acc, w[0], f);
#pragma unroll
                    for (int m = 1; m < kW; ++m) accumulate<V>(acc, w[m], win[m - 1]);
                    store_pack<IoT, V>(out + (i0 + i) * ostride, finished<IoT, V>(acc, a.activation));
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) {
#pragma unroll
                        for (int m = kPast - 1; m > 0; --m) win[m][j] = win[m - 1][j];
                        win[0][j] = f[j];
                    }
                }
            } else {
#pragma unroll
                for (int m = 0; m < kPast; ++m) widen<IoT, V>(now[kGroup - 1 - m], win[m]);
            }
            // the group is in registers: its place takes the one kDepth groups on
            if constexpr (kAsync) {
                load_group(i0 + kDepth * kGroup, stage);
                stage = stage + 1 == kDepth ? 0 : stage + 1;
            }
        }
        if (!(what & kSlides)) {
            for (int s0 = i0; s0 < min(i0 + kGroup, nt); s0 += kSlow) {
                Pack<IoT, V> tap[kSlow][kM];
#pragma unroll
                for (int i = 0; i < kSlow; ++i) {
                    const Token k = token[s0 + i];
#pragma unroll
                    for (int m = 0; m < kM; ++m) {
                        tap[i][m] = Pack<IoT, V>{};
                        if (m >= W || k.local < 0) continue;
                        const IoT *src = nullptr;
                        if (m <= k.local) {
                            src = x + (int64_t)(s0 + i - m) * a.xbc_stride;
                        } else if (m <= k.past && k.slot >= 0) {
                            int row = k.row - m;
                            if (row < 0) row += a.conv_rows;
                            src = ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels;
                        }
                        if (src) tap[i][m] = load_pack<IoT, V>(src);
                    }
                }
#pragma unroll
                for (int i = 0; i < kSlow; ++i) {
                    if (token[s0 + i].local < 0) continue;
                    float2 acc[kPairs];
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) acc[j] = bias[j];
#pragma unroll
                    for (int m = 0; m < kM; ++m)
                        if (m < W) {
                            float2 f[kPairs];
                            widen<IoT, V>(tap[i][m], f);
                            accumulate<V>(acc, w[m], f);
                        }
                    store_pack<IoT, V>(out + (s0 + i) * ostride, finished<IoT, V>(acc, a.activation));
                }
            }
        }
        if (what & kKeeps) {
            for (int i = i0; i < min(i0 + kGroup, nt); ++i) {
                if (!keep[i]) continue;
                const Token k = token[i];
                store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + k.row) * a.channels,
                                   load_pack<IoT, V>(x + i * a.xbc_stride));
            }
        }
    }

    if constexpr (kAsync) wait_async<0>();
    // the end of the sequence that begins in this tile and passes it
    const int s = tail_seq;
    if (s >= 0) {
        const Token k = token[nt - 1];
        const int64_t e = (int64_t)a.cu_seqlens[s + 1] - t0;       // tokens from the tile's first
        for (int64_t i = max((int64_t)nt, e - (W - 1)); i < e; ++i) {
            const int row = (int)((k.row + (i - (nt - 1))) % a.conv_rows);
            store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels,
                               load_pack<IoT, V>(x + i * a.xbc_stride));
        }
    }
}

template <typename IoT, int V>
cudaError_t launch(const ssd_conv_params &p, cudaStream_t stream) {
    const int ctiles = (p.channels + kThreads * V - 1) / (kThreads * V), dt = p.dt != nullptr ? 1 : 0;
    // long tiles read fewer tokens twice; short ones fill the GPU
    int tile = kMaxTile;
    while (tile > kGroup && (p.total_tokens + tile - 1) / tile * ctiles < 152 * 8) tile /= 2;
    const int64_t tiles = (p.total_tokens + tile - 1) / tile;
    if (tiles > 0x7fffffff || ctiles + dt > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles, (unsigned)(ctiles + dt));
    switch (p.width) {
        case 2: conv_kernel<IoT, V, 2><<<grid, kThreads, 0, stream>>>(p, tile, dt); break;
        case 3: conv_kernel<IoT, V, 3><<<grid, kThreads, 0, stream>>>(p, tile, dt); break;
        case 4: conv_kernel<IoT, V, 4><<<grid, kThreads, 0, stream>>>(p, tile, dt); break;
        default: conv_kernel<IoT, V, 0><<<grid, kThreads, 0, stream>>>(p, tile, dt);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_conv(const ssd_conv_params &p, cudaStream_t stream) {
    const int io = p.io_dtype == SSD_F32 ? 4 : 2;
    const int rest = p.channels - p.split0 - p.split1;
    auto can = [&](int v) {
        const size_t bytes = (size_t)v * io;
        return p.channels % v == 0 && p.xbc_stride % v == 0 && p.split0 % v == 0 && p.split1 % v == 0 &&
               rest % v == 0 && aligned_to(p.xbc, bytes) && aligned_to(p.conv_cache, bytes) &&
               aligned_to(p.out0, bytes) && aligned_to(p.out1, bytes) && aligned_to(p.out2, bytes) &&
               aligned_to(p.weight, 16) && aligned_to(p.bias, bytes);
    };
    if (p.io_dtype == SSD_F32)
        return can(4) ? launch<float, 4>(p, stream) : can(2) ? launch<float, 2>(p, stream) : launch<float, 1>(p, stream);
    return can(4)   ? launch<__nv_bfloat16, 4>(p, stream)
           : can(2) ? launch<__nv_bfloat16, 2>(p, stream)
                    : launch<__nv_bfloat16, 1>(p, stream);
}

}  // namespace ssd
