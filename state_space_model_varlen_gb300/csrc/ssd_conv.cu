// Short causal convolution of packed prompts, split into the scan's inputs.
//
//   u_t[c] = act(bias[c] + sum_{k < W} w[c, W-1-k] xbc_{t-k}[c])
//
// Each value is read once and written once: the kernel is bound by HBM.  A CTA
// owns a tile of tokens and of channels; a thread owns V neighbouring channels
// (16 bytes) and walks the tile's tokens with the last W - 1 inputs in
// registers, so a tile reads W - 1 tokens more than it writes.
//
// Sequence boundaries are worked out once per CTA: every thread looks at some
// of the sequences and marks the tile's tokens in shared memory; the walk then
// reads one record per token.
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
constexpr int kMaxTile = 32;       // tokens of a tile

struct Token {
    int local;      // token of its sequence, -1: no valid sequence
    int row;        // its row of the ring
    int slot;       // -1: no cache
    int past;       // min(position, W - 1) << 1 | this token is written to the ring here
};

template <typename IoT, int V, int kW>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ssd_conv_params a, int tile, int ctiles) {
    __shared__ int seq_of[kMaxTile];
    __shared__ Token token[kMaxTile];
    __shared__ int tail_seq;
    const int W = kW ? kW : a.width;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)min((int64_t)tile, a.total_tokens - t0);
    const int ct = blockIdx.y;

    // the last column of CTAs widens dt
    if (ct == ctiles) {
        const IoT *dt = static_cast<const IoT *>(a.dt);
        for (int i = threadIdx.x; i < nt * a.nheads; i += kThreads) {
            const int64_t t = t0 + i / a.nheads;
            const int h = i % a.nheads;
            a.out_dt[t * a.nheads + h] = to_float(dt[t * a.dt_stride + h]);
        }
        return;
    }

    // ---- the tile's tokens -------------------------------------------------
    if (threadIdx.x < tile) seq_of[threadIdx.x] = -1;
    if (threadIdx.x == 0) tail_seq = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < a.num_seqs; s += kThreads) {
        const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
        if (b < 0 || e < b || e > a.total_tokens) {
            if (t0 == 0 && ct == 0 && a.device_status) atomicOr(a.device_status, SSD_DEV_BAD_SEQLENS);
            continue;
        }
        const int64_t lo = max(b, t0), hi = min(e, t0 + nt);
        for (int64_t t = lo; t < hi; ++t) seq_of[t - t0] = s;
    }
    __syncthreads();
    if (threadIdx.x < nt) {
        const int s = seq_of[threadIdx.x];
        Token k = {-1, 0, -1, 0};
        if (s >= 0) {
            const int64_t b = a.cu_seqlens[s], e = a.cu_seqlens[s + 1];
            const int64_t local = t0 + threadIdx.x - b;
            const int start = a.start_pos ? a.start_pos[s] : 0;
            int slot = -1;
            bool ok = true;
            if (a.conv_cache != nullptr) {
                slot = a.slot_idx[s * (a.slot_idx_stride ? a.slot_idx_stride : 1)];
                ok = slot >= 0 && slot < a.num_slots;
                if (!ok && local == 0 && ct == 0 && a.device_status) atomicOr(a.device_status, SSD_DEV_BAD_SLOT);
            }
            if (start < 0) {
                ok = false;
                if (local == 0 && ct == 0 && a.device_status) atomicOr(a.device_status, SSD_DEV_BAD_POS);
            }
            if (ok) {
                const int64_t pos = start + local;
                const bool begins_here = b >= t0;
                k.local = (int)min(local, (int64_t)0x7fffffff);
                k.slot = slot;
                k.row = slot >= 0 ? (int)(pos % a.conv_rows) : 0;
                const bool keep = slot >= 0 && begins_here && t0 + threadIdx.x >= e - (W - 1);
                k.past = (int)min(pos, (int64_t)(W - 1)) << 1 | (keep ? 1 : 0);
                // the tile's last sequence goes on after it: its end is kept below
                if (slot >= 0 && begins_here && threadIdx.x == nt - 1 && e > t0 + nt) tail_seq = s;
            }
        }
        token[threadIdx.x] = k;
    }
    __syncthreads();

    const int c = (ct * kThreads + threadIdx.x) * V;
    if (c >= a.channels) return;
    const IoT *x = static_cast<const IoT *>(a.xbc) + c;
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

    constexpr int kM = kW ? kW : SSD_CONV_MAX_WIDTH;
    float w[kM][V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bias[j] = a.bias ? to_float(static_cast<const IoT *>(a.bias)[c + j]) : 0.f;
#pragma unroll
        for (int k = 0; k < kM; ++k)     // w[k]: the tap of the token k before
            w[k][j] = k < W ? to_float(static_cast<const IoT *>(a.weight)[(int64_t)(c + j) * W + (W - 1 - k)]) : 0.f;
    }

    // win[k]: the input k tokens before the current one
    float win[kM][V];
#pragma unroll
    for (int k = 0; k < kM; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) win[k][j] = 0.f;

    for (int i = 0; i < nt; ++i) {
        const Token k = token[i];
        if (k.local < 0) continue;
        const int64_t t = t0 + i;
        const Pack<IoT, V> now = load_pack<IoT, V>(x + t * a.xbc_stride);
#pragma unroll
        for (int m = kM - 1; m > 0; --m)
#pragma unroll
            for (int j = 0; j < V; ++j) win[m][j] = win[m - 1][j];
#pragma unroll
        for (int j = 0; j < V; ++j) win[0][j] = to_float(now.v[j]);
        if (k.local == 0 || i == 0) {
            // the window's past: from the sequence's tokens, the ring, or zero
#pragma unroll
            for (int m = 1; m < kM; ++m) {
                if (m >= W) break;
#pragma unroll
                for (int j = 0; j < V; ++j) win[m][j] = 0.f;
                const IoT *src = nullptr;
                if (m <= k.local) {
                    src = x + (t - m) * a.xbc_stride;
                } else if (m <= (k.past >> 1) && k.slot >= 0) {
                    int row = k.row - m;
                    if (row < 0) row += a.conv_rows;
                    src = ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels;
                }
                if (src) {
                    const Pack<IoT, V> p = load_pack<IoT, V>(src);
#pragma unroll
                    for (int j = 0; j < V; ++j) win[m][j] = to_float(p.v[j]);
                }
            }
        }
        Pack<IoT, V> u;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float acc = bias[j];
#pragma unroll
            for (int m = 0; m < kM; ++m)
                if (m < W) acc = fmaf(w[m][j], win[m][j], acc);
            u.v[j] = from_float<IoT>(a.activation ? silu(acc) : acc);
        }
        store_pack<IoT, V>(out + t * ostride, u);
        if (k.past & 1) store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + k.row) * a.channels, now);
    }

    // the end of the sequence that begins in this tile and passes it
    const int s = tail_seq;
    if (s >= 0) {
        const Token k = token[nt - 1];
        const int64_t e = a.cu_seqlens[s + 1];
        for (int64_t t = max(t0 + nt, e - (W - 1)); t < e; ++t) {
            const int row = (int)((k.row + (t - (t0 + nt - 1))) % a.conv_rows);
            store_pack<IoT, V>(ring + ((int64_t)k.slot * a.conv_rows + row) * a.channels,
                               load_pack<IoT, V>(x + t * a.xbc_stride));
        }
    }
}

template <typename IoT, int V>
cudaError_t launch(const ssd_conv_params &p, cudaStream_t stream) {
    const int tile = kMaxTile;
    const int64_t tiles = (p.total_tokens + tile - 1) / tile;
    const int ctiles = (p.channels + kThreads * V - 1) / (kThreads * V);
    if (tiles > 0x7fffffff || ctiles + 1 > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles, (unsigned)(ctiles + (p.dt != nullptr ? 1 : 0)));
    if (p.width == 4)
        conv_kernel<IoT, V, 4><<<grid, kThreads, 0, stream>>>(p, tile, ctiles);
    else
        conv_kernel<IoT, V, 0><<<grid, kThreads, 0, stream>>>(p, tile, ctiles);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_conv(const ssd_conv_params &p, cudaStream_t stream) {
    const int io = p.io_dtype == SSD_F32 ? 4 : 2, v = 16 / io;
    const int rest = p.channels - p.split0 - p.split1;
    const bool wide = p.channels % v == 0 && p.xbc_stride % v == 0 && p.split0 % v == 0 && p.split1 % v == 0 &&
                      rest % v == 0 && aligned_to(p.xbc, 16) && aligned_to(p.conv_cache, 16) &&
                      aligned_to(p.out0, 16) && aligned_to(p.out1, 16) && aligned_to(p.out2, 16);
    if (p.io_dtype == SSD_F32) return wide ? launch<float, 4>(p, stream) : launch<float, 1>(p, stream);
    return wide ? launch<__nv_bfloat16, 8>(p, stream) : launch<__nv_bfloat16, 1>(p, stream);
}

}  // namespace ssd
