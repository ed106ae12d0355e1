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
// Sequence boundaries are worked out once per CTA, while the first groups'
// inputs are on their way: every thread looks at some of the sequences, and
// those that meet the tile leave a record at their first token in it.  A group
// whose tokens all have their W - 1 predecessors in this call slides the
// window.  In any other, batches of short sequences copy what the tokens lack
// from the ring all at once (kShort); batches of long ones, where such groups
// are few, load every tap from where it lies, two tokens at a time, which
// leaves the shared memory to the inputs.
//
// The convolution cache is updated in place, so one thread does all that a
// sequence reads and writes of a channel's ring: the CTA whose tile holds the
// sequence's first token.  It computes the sequence's first W - 1 tokens, the
// only ones that need the ring, also where they pass the tile's end (the next
// tile leaves them out), and afterwards writes the sequence's last inputs,
// also where those lie in later tiles.
//
// Measured: 61,773 tokens of 10,240 bf16 channels in 32 prompts 399 us, 6.5 TB/s
// (95 % of the copy rate); 2,232 tokens 22.4 us (floor 13.7); 200 single tokens
// and a chunk of 1,111, 5,376 channels, 16.8 us (floor 4.2), where each group
// with sequence starts, three of a tile, is a memory round trip of its own.
#include <algorithm>

#include "ssd_mixer_common.cuh"
#include "ssd_mixer_internal.h"

namespace ssd {
namespace {

constexpr int kThreads = 128;       // of a CTA at most: fewer where the channels do not fill them
constexpr int kMaxTile = 64;       // tokens of a tile
constexpr int kRecords = kMaxTile + SSD_CONV_MAX_WIDTH;       // and those after it that it may take over
constexpr int kGroup = 8;          // tokens whose inputs are loaded together
constexpr int kSlow = 2;           // tokens whose taps are loaded together at a boundary

struct Token {
    int local;      // token of its sequence, -1: none of this CTA's
    int row;        // its row of the ring
    int slot;       // -1: no cache
    int past;       // min(position, W - 1)
};
struct Sequence {
    int64_t begin, end;
    int start, slot;    // slot -1: no cache
};
constexpr int kSlides = 1, kKeeps = 2;      // of a group: every token has its window here; some go to the ring

// Sequence s as its metadata has it, and the status bits of what is wrong there.
__device__ __forceinline__ Sequence look_up(const ssd_conv_params &a, int s) {
    Sequence q = {a.cu_seqlens[s], a.cu_seqlens[s + 1], 0, -1};
    if (a.start_pos) q.start = a.start_pos[s];
    if (a.conv_cache) q.slot = a.slot_idx[s * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
    return q;
}
__device__ __forceinline__ int faults(const ssd_conv_params &a, const Sequence &q) {
    if (q.begin < 0 || q.end < q.begin || q.end > a.total_tokens) return SSD_DEV_BAD_SEQLENS;
    if (q.end > q.begin && a.conv_cache && (q.slot < 0 || q.slot >= a.num_slots)) return SSD_DEV_BAD_SLOT;
    return q.end > q.begin && q.start < 0 ? SSD_DEV_BAD_POS : 0;
}

// dt of the tile's tokens that are some valid sequence's, widened to fp32.  The
// first tokens' loads are on their way while the sequences are looked up.
template <typename IoT>
__device__ __forceinline__ void widen_dt(const ssd_conv_params &a, int64_t t0, int nt) {
    __shared__ uint32_t live[kMaxTile / 32];
    const IoT *dt = static_cast<const IoT *>(a.dt) + t0 * a.dt_stride;
    float v[kGroup];
    auto load = [&](int h, int i) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (i + j < nt) v[j] = to_float(dt[(i + j) * a.dt_stride + h]);
    };
    if ((int)threadIdx.x < a.nheads) load(threadIdx.x, 0);
    if (threadIdx.x < kMaxTile / 32) live[threadIdx.x] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.num_seqs; s += blockDim.x) {
        const Sequence q = look_up(a, s);
        const int first = (int)max(q.begin - t0, (int64_t)0), end = (int)min(q.end - t0, (int64_t)nt);
        if (faults(a, q) || end <= first) continue;
        for (int w = first / 32; w * 32 < end; ++w) {
            const int lo = max(first - w * 32, 0), n = min(end - w * 32, 32) - lo;
            atomicOr(&live[w], (0xffffffffu >> (32 - n)) << lo);
        }
    }
    __syncthreads();
    for (int h = threadIdx.x; h < a.nheads; h += blockDim.x) {
        for (int i = 0; i < nt; i += kGroup) {
            if (i > 0 || h >= (int)blockDim.x) load(h, i);
            const uint32_t mask = live[i / 32] >> (i % 32);
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (mask >> j & 1) a.out_dt[(t0 + i + j) * a.nheads + h] = v[j];
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
constexpr int kMinCtas = kW == 0 ? 3 : 5;

// kW: the width, or 0 for one that only a.width tells (then no group slides).
// kSplit: only the rows of xbc are not aligned to V elements: they are loaded
// one element at a time, everything else V together.
template <typename IoT, int V, int kW, bool kShort, bool kSplit>
__global__ void __launch_bounds__(kThreads, kMinCtas<IoT, V, kW>) conv_kernel(const ssd_conv_params a, int tile, int dt_column) {
    __shared__ Sequence sequence[kMaxTile];        // at the sequence's first token in the tile
    __shared__ uint32_t firsts[kMaxTile / 32];      // where there are any
    __shared__ Token token[kRecords];
    __shared__ uint8_t keep[kMaxTile];             // the token goes to the ring here
    __shared__ int group[kMaxTile / kGroup];
    __shared__ int after;                          // tokens after the tile that are this CTA's
    __shared__ int64_t tail;                       // where that sequence ends, from the tile's first token; 0: none
    constexpr int kM = kW ? kW : SSD_CONV_MAX_WIDTH;
    constexpr int kPast = kW > 1 ? kW - 1 : 1;      // inputs a sliding window keeps
    constexpr int kPairs = (V + 1) / 2;
    // groups copied ahead; two-byte shares are loaded one group ahead instead
    constexpr int kBytes = V * (int)sizeof(IoT);
    constexpr bool kAsync = kBytes >= 4 && kW > 1 && !kSplit;
    constexpr int kDepth = kBytes < 8 ? 4 : kShort ? 2 : 3;
    __shared__ Pack<IoT, V> s_x[kAsync ? kDepth * kGroup * kThreads : 1];
    __shared__ Pack<IoT, V> s_old[kAsync && kShort ? kGroup * kPast * kThreads : 1];
    await_previous();
    const int W = kW ? kW : a.width;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)min((int64_t)tile, a.total_tokens - t0);
    const int ct = (int)blockIdx.y - dt_column;
    if (ct < 0) {
        widen_dt<IoT>(a, t0, nt);
        return;
    }
    const bool reporter = ct == 0 && a.device_status != nullptr;

    // ---- every load that depends on nothing: sequences, inputs, weights -----
    Sequence seq{};
    if ((int)threadIdx.x < a.num_seqs) seq = look_up(a, threadIdx.x);
    const int c = (ct * blockDim.x + threadIdx.x) * V;
    const bool mine = c < a.channels;
    const IoT *x = static_cast<const IoT *>(a.xbc) + t0 * a.xbc_stride + c;    // of the tile's first token
    Pack<IoT, V> next[kGroup], prev[kPast];
    auto load_x = [](const IoT *src) {
        if constexpr (kSplit) {
            Pack<IoT, V> p;
#pragma unroll
            for (int j = 0; j < V; ++j) p.v[j] = src[j];
            return p;
        } else {
            return load_pack<IoT, V>(src);
        }
    };
    auto load_group = [&](int i0, int stage) {
        const IoT *src = x + i0 * a.xbc_stride;
        if (mine && i0 + kGroup <= nt) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j, src += a.xbc_stride) {
                if constexpr (kAsync) copy_async<kBytes>(&s_x[(stage * kGroup + j) * kThreads + threadIdx.x], src, true);
                else next[j] = load_x(src);
            }
        } else if (mine && i0 < nt) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j, src += a.xbc_stride) {
                const bool live = i0 + j < nt;
                if constexpr (kAsync)
                    copy_async<kBytes>(&s_x[(stage * kGroup + j) * kThreads + threadIdx.x],
                                       live ? src : static_cast<const IoT *>(a.xbc), live);
                else if (live)
                    next[j] = load_x(src);
            }
        }
        if constexpr (kAsync) commit_async();
    };
    if constexpr (kW > 1) {
#pragma unroll
        for (int d = 0; d < (kAsync ? kDepth : 1); ++d) load_group(d * kGroup, d);
#pragma unroll
        for (int m = 1; m < kW; ++m) {
            prev[m - 1] = Pack<IoT, V>{};
            if (mine && t0 >= m) prev[m - 1] = load_x(x - m * a.xbc_stride);
        }
    }

    Pack<IoT, V * kM> pw{};
    Pack<IoT, V> pb{};
    if constexpr (kW > 0 && V > 1) {
        if (mine) {
            pw = load_pack<IoT, V * kM>(static_cast<const IoT *>(a.weight) + (int64_t)c * kM);
            if (a.bias) pb = load_pack<IoT, V>(static_cast<const IoT *>(a.bias) + c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (mine && a.bias) pb.v[j] = static_cast<const IoT *>(a.bias)[c + j];
#pragma unroll
            for (int k = 0; k < kM; ++k)        // as a width of kM with leading zeros
                if (mine && k < W)
                    pw.v[j * kM + kM - 1 - k] = static_cast<const IoT *>(a.weight)[(int64_t)(c + j) * W + (W - 1 - k)];
        }
    }

    // ---- the tile's tokens -------------------------------------------------
    static_assert(kMaxTile / kGroup <= 32 && kMaxTile / 32 <= 32, "the smallest CTA has a warp");
    if (threadIdx.x < kMaxTile / 32) firsts[threadIdx.x] = 0;
    if (threadIdx.x < kMaxTile / kGroup) group[threadIdx.x] = kW > 1 ? kSlides : 0;
    if (threadIdx.x == 0) tail = after = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.num_seqs; s += blockDim.x) {
        const Sequence q = s == (int)threadIdx.x ? seq : look_up(a, s);
        const int bad = faults(a, q);
        if (bad) {
            if (blockIdx.x == 0 && reporter) atomicOr(a.device_status, bad);
        } else if (q.begin < t0 + nt && q.end > t0 && q.end > q.begin) {
            const int first = (int)(max(q.begin, t0) - t0);
            sequence[first] = q;
            atomicOr(&firsts[first / 32], 1u << (first % 32));
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRecords; i += blockDim.x) {
        // the last first token up to this one (a token after the tile: up to the tile's last)
        const int to = min(i, nt - 1);
        const uint32_t below = firsts[to / 32] & (0xffffffffu >> (31 - to % 32));
        int first = below ? (to & ~31) + 31 - __clz(below) : -1;
        for (int word = to / 32 - 1; first < 0 && word >= 0; --word)
            if (firsts[word]) first = word * 32 + 31 - __clz(firsts[word]);
        Token k = {-1, 0, -1, 0};
        bool kept = false;
        if (first >= 0 && sequence[first].end > t0 + i) {
            const Sequence q = sequence[first];
            const int64_t local = t0 + i - q.begin, pos = q.start + local;
            const bool begins_here = q.begin >= t0;
            if (i < nt ? begins_here || local >= W - 1 : begins_here && local < W - 1) {
                k.local = (int)min(local, (int64_t)0x7fffffff);
                k.slot = q.slot;
                k.row = q.slot >= 0 ? (int)(pos % a.conv_rows) : 0;
                k.past = (int)min(pos, (int64_t)(W - 1));
                kept = i < nt && q.slot >= 0 && begins_here && t0 + i >= q.end - (W - 1);
                // the tile's last sequence goes on after it: its end is kept below
                if (q.slot >= 0 && begins_here && i == nt - 1 && q.end > t0 + nt) tail = q.end - t0;
                if (i >= nt) atomicMax(&after, i + 1 - nt);
            }
        }
        token[i] = k;
        if (i < kMaxTile) {
            keep[i] = kept;
            if (k.local < W - 1) atomicAnd(&group[i / kGroup], ~kSlides);
            if (kept) atomicOr(&group[i / kGroup], kKeeps);
        }
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
#pragma unroll
    for (int j = 0; j < V; ++j) {
        (j & 1 ? bias[j / 2].y : bias[j / 2].x) = to_float(pb.v[j]);
#pragma unroll
        for (int k = 0; k < kM; ++k)
            (j & 1 ? w[k][j / 2].y : w[k][j / 2].x) = to_float(pw.v[j * kM + kM - 1 - k]);
    }
    // the tokens from .. to - 1, every tap from where it lies
    auto boundary = [&](int from, int to) {
#pragma unroll 1
        for (int s0 = from; s0 < to; s0 += kSlow) {
            Pack<IoT, V> tap[kSlow][kM];
#pragma unroll
            for (int i = 0; i < kSlow; ++i) {
                const Token k = token[s0 + i];
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    tap[i][m] = Pack<IoT, V>{};
                    if (m >= W || k.local < 0 || s0 + i >= to) continue;
                    if (m <= k.local) {
                        tap[i][m] = load_x(x + (int64_t)(s0 + i - m) * a.xbc_stride);
                    } else if (m <= k.past && k.slot >= 0) {
                        int row = k.row - m;
                        if (row < 0) row += a.conv_rows;
                        tap[i][m] = load_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kSlow; ++i) {
                if (token[s0 + i].local < 0 || s0 + i >= to) continue;
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
    };

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
            // a token's value from its input and the W - 1 before it, and the window moved on
            auto one = [&](int i, bool write, auto before) {
                float2 acc[kPairs], f[kPairs];
                widen<IoT, V>(now[i], f);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) acc[j] = bias[j];
                accumulate<V>(acc, w[0], f);
#pragma unroll
                for (int m = 1; m < kW; ++m) {
                    float2 g[kPairs];
                    before(m, g);
                    accumulate<V>(acc, w[m], g);
                }
                if (write) store_pack<IoT, V>(out + (i0 + i) * ostride, finished<IoT, V>(acc, a.activation));
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
#pragma unroll
                    for (int m = kPast - 1; m > 0; --m) win[m][j] = win[m - 1][j];
                    win[0][j] = f[j];
                }
            };
            if (what & kSlides) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i)
                    one(i, true, [&](int m, float2 (&g)[kPairs]) {
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) g[j] = win[m - 1][j];
                    });
            } else if constexpr (!kShort) {
                boundary(i0, min(i0 + kGroup, nt));
#pragma unroll
                for (int m = 0; m < kPast; ++m) widen<IoT, V>(now[kGroup - 1 - m], win[m]);
            } else {
                Pack<IoT, V> old[kAsync ? 1 : kGroup][kPast];
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const Token k = token[i0 + i];
#pragma unroll
                    for (int m = 1; m < kW; ++m) {
                        const bool live = k.local >= 0 && m > k.local && m <= k.past && k.slot >= 0;
                        int row = k.row - m;
                        if (row < 0) row += a.conv_rows;
                        const IoT *src = live ? ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels
                                              : static_cast<const IoT *>(a.xbc);
                        if constexpr (kAsync) {
                            copy_async<kBytes>(&s_old[(i * kPast + m - 1) * kThreads + threadIdx.x], src, live);
                        } else {
                            old[i][m - 1] = Pack<IoT, V>{};
                            if (live) old[i][m - 1] = load_pack<IoT, V>(src);
                        }
                    }
                }
                if constexpr (kAsync) {
                    commit_async();
                    wait_async<0>();
                }
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const int local = token[i0 + i].local;
                    one(i, local >= 0, [&](int m, float2 (&g)[kPairs]) {
                        widen<IoT, V>(kAsync ? s_old[(i * kPast + m - 1) * kThreads + threadIdx.x] : old[kAsync ? 0 : i][m - 1], g);
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) {
                            g[j].x = m <= local ? win[m - 1][j].x : g[j].x;
                            if (V > 1) g[j].y = m <= local ? win[m - 1][j].y : g[j].y;
                        }
                    });
                }
            }
            // after the group's taps are read: a short sequence writes rows that it read
            if (what & kKeeps) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const Token k = token[i0 + i];
                    if (keep[i0 + i])
                        store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + k.row) * a.channels, now[i]);
                }
            }
            // the group is in registers: its place takes the one kDepth groups on
            if constexpr (kAsync) {
                load_group(i0 + kDepth * kGroup, stage);
                stage = stage + 1 == kDepth ? 0 : stage + 1;
            }
        }
        if constexpr (kW <= 1) boundary(i0, min(i0 + kGroup, nt));
        if (kW <= 1 && (what & kKeeps)) {
            for (int i = i0; i < min(i0 + kGroup, nt); ++i) {
                if (!keep[i]) continue;
                const Token k = token[i];
                store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + k.row) * a.channels,
                                   load_x(x + i * a.xbc_stride));
            }
        }
    }

    if constexpr (kAsync) wait_async<0>();
    boundary(nt, nt + after);
    // the end of the sequence that begins in this tile and passes it
    const int64_t e = tail;
    if (e > 0) {
        const Token k = token[nt - 1];
        const int64_t i0 = max((int64_t)nt, e - (W - 1));
        Pack<IoT, V> last[kM];
#pragma unroll
        for (int m = 0; m < kM; ++m)
            if (i0 + m < e) last[m] = load_x(x + (i0 + m) * a.xbc_stride);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            if (i0 + m >= e) break;
            const int row = (int)((k.row + (i0 + m - (nt - 1))) % a.conv_rows);
            store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels, last[m]);
        }
    }
}

template <typename IoT, int V, bool kSplit>
cudaError_t launch(const ssd_conv_params &p, cudaStream_t stream) {
    const int lanes = (p.channels + V - 1) / V, ctiles = (lanes + kThreads - 1) / kThreads, dt = p.dt != nullptr ? 1 : 0;
    const int threads = ((lanes + ctiles - 1) / ctiles + 31) / 32 * 32;
    // mean length below 64: many groups hold a sequence's first token (201
    // sequences, 1,311 tokens of 5,376 channels: 16.8 us so, 22.3 the other way; 61,773
    // tokens of 10,240 channels in 32 sequences: 492 and 399)
    const bool brief = !kSplit && p.total_tokens < 64LL * p.num_seqs;
    // the tile whose waves of CTAs take the least, a CTA's own start counted as
    // 24 tokens: long tiles for long batches, one wave of shorter ones below that
    int tile = kGroup;
    int64_t least = INT64_MAX;
    // what the registers leave room for, at most what the shared memory does: eight,
    // with the ring's share of a group five (44 of 228 KB each)
    const int64_t resident = 152LL * std::min(brief && p.width == 4 ? 5 : 8, kMinCtas<IoT, V, 4> * kThreads / threads);
    for (int t = kGroup; t <= kMaxTile; t += kGroup) {
        const int64_t ctas = (p.total_tokens + t - 1) / t * ctiles, cost = (ctas + resident - 1) / resident * (t + 24);
        if (cost <= least) {
            least = cost;
            tile = t;
        }
    }
    const int64_t tiles = (p.total_tokens + tile - 1) / tile;
    if (tiles > 0x7fffffff || ctiles + dt > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles, (unsigned)(ctiles + dt));
    auto run = [&](auto kernel) { return enqueue(kernel, grid, threads, stream, p, tile, dt); };
    switch (p.width) {
        case 2: return brief ? run(conv_kernel<IoT, V, 2, !kSplit, kSplit>) : run(conv_kernel<IoT, V, 2, false, kSplit>);
        case 3: return brief ? run(conv_kernel<IoT, V, 3, !kSplit, kSplit>) : run(conv_kernel<IoT, V, 3, false, kSplit>);
        case 4: return brief ? run(conv_kernel<IoT, V, 4, !kSplit, kSplit>) : run(conv_kernel<IoT, V, 4, false, kSplit>);
    }
    return run(conv_kernel<IoT, V, 0, false, kSplit>);
}

}  // namespace

cudaError_t launch_conv(const ssd_conv_params &p, cudaStream_t stream) {
    const int io = p.io_dtype == SSD_F32 ? 4 : 2;
    const int rest = p.channels - p.split0 - p.split1;
    auto rest_can = [&](int v) {
        const size_t bytes = (size_t)v * io;
        return p.channels % v == 0 && p.split0 % v == 0 && p.split1 % v == 0 && rest % v == 0 &&
               aligned_to(p.conv_cache, bytes) && aligned_to(p.out0, bytes) && aligned_to(p.out1, bytes) &&
               aligned_to(p.out2, bytes) && aligned_to(p.weight, 16) && aligned_to(p.bias, bytes);
    };
    auto can = [&](int v) { return rest_can(v) && p.xbc_stride % v == 0 && aligned_to(p.xbc, (size_t)v * io); };
    // eight bytes a thread: more would not leave room for the ring's share of a group
    if (p.io_dtype == SSD_F32) return can(2) ? launch<float, 2, false>(p, stream) : launch<float, 1, false>(p, stream);
    if (can(4)) return launch<__nv_bfloat16, 4, false>(p, stream);
    if (can(2)) return launch<__nv_bfloat16, 2, false>(p, stream);
    if (rest_can(4)) return launch<__nv_bfloat16, 4, true>(p, stream);
    return rest_can(2) ? launch<__nv_bfloat16, 2, true>(p, stream) : launch<__nv_bfloat16, 1, false>(p, stream);
}

}  // namespace ssd
