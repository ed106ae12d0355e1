// Verification of drafted tokens: the first draft of a window that does not stand,
// and the token in its place (or behind the last draft).
//
//   draft i stands while u_i q_i(d_i) < p_i(d_i)
//   w = max(p - q, 0) of the row where it stopped;  new = the lowest t with cum_t > u cum_V
//
// The sums decide which whole number comes out, so they are kept to about 48 bits:
// pairs of floats whose additions keep what rounding drops (Knuth's two-sum; for
// p - q with p > q Dekker's shorter form), and doubles where there are few terms.
// In doubles alone the additions of a 128-window batch would take longer than its
// reads (two fp64 operations a clock and SM).  Bound by HBM: one row of p, and one
// of q where a draft fell.
#include "ssd_layer_internal.h"
#include "ssd_mixer_common.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

// s + c, s the rounded sum
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ void add(float v, float rest) {
        const float t = s + v, b = t - s;
        c += ((s - (t - b)) + (v - b)) + rest;
        s = t;
    }
    __device__ double value() const { return (double)s + (double)c; }
};

__device__ __forceinline__ double warp_total(const Sum &a) {
    double v = a.value();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Where w comes from: the target's row, less the draft's row or what was drafted.
template <typename T> struct Weights {
    const T *p, *q;
    int without;                // token whose weight is 0, or -1
    // w of token t as a rounded value and what its rounding dropped
    __device__ float2 operator()(int t) const {
        const float a = to_float(p[t]), b = q ? to_float(q[t]) : 0.f;
        const float d = a - b;
        // 0 < d finite: a > b; b < 0 or not finite does not come with probabilities
        return d > 0.f && d < __int_as_float(0x7f800000) && t != without ? make_float2(d, (a - d) - b) : make_float2(0.f, 0.f);
    }
};

template <typename T> struct Window {
    int a, k, n;                // first token; drafts; drafts that stand
    bool live;
    Weights<T> w;
};

__device__ __forceinline__ void flag(int32_t *status, int bit) {
    if (status) atomicOr(status, bit);
}

template <typename T> __global__ void __launch_bounds__(kThreads) verify_kernel(const ssd_verify_params a) {
    __shared__ Window<T> win;
    __shared__ double part[kWarps];
    __shared__ int found;
    await_previous();
    const int s = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = a.vocab;
    const T *const target = static_cast<const T *>(a.target_probs), *const draft = static_cast<const T *>(a.draft_probs);
    if (warp == 0) {
        const int64_t first = a.cu_seqlens[s], end = a.cu_seqlens[s + 1];
        const int64_t k = end - first - 1, d0 = first - s;
        bool ok = true;
        if (first < 0 || end < first || end > a.total_tokens || (k > 0 && (d0 < 0 || d0 + k > a.num_drafts))) {
            if (lane == 0) flag(a.device_status, SSD_DEV_BAD_SEQLENS);
            ok = false;
        }
        ok = ok && k >= 0;
        int n = 0;
        for (int base = 0; ok && base < k; base += 32) {
            const int i = base + lane;
            bool stands = true, bad = false;
            if (i < k) {
                const int tok = a.tokens[first + i + 1];
                bad = tok < 0 || tok >= V;
                if (!bad) {
                    const double q = draft ? (double)to_float(draft[(d0 + i) * a.draft_stride + tok]) : 1.0;
                    const double p = (double)to_float(target[(first + i) * a.target_stride + tok]);
                    stands = (double)fminf(fmaxf(a.accept_u[d0 + i], 0.f), 1.f) * q < p;
                }
            }
            const uint32_t stop = __ballot_sync(0xffffffffu, bad || !stands), wrong = __ballot_sync(0xffffffffu, bad);
            if (stop) {
                const int at = __ffs(stop) - 1;
                n = base + at;
                if (wrong >> at & 1) {
                    if (lane == 0) flag(a.device_status, SSD_DEV_BAD_TOKEN);
                    ok = false;
                }
                break;
            }
            n = (int)min((int64_t)base + 32, k);
        }
        if (lane == 0) {
            win.live = ok;
            win.a = (int)first;
            win.k = (int)k;
            win.n = n;
            if (ok) {
                win.w.p = target + (first + n) * a.target_stride;
                win.w.q = draft && n < k ? draft + (d0 + n) * a.draft_stride : nullptr;
                win.w.without = !draft && n < k ? a.tokens[first + n + 1] : -1;
            }
            found = -1;
        }
    }
    __syncthreads();
    if (!win.live) return;
    Weights<T> w = win.w;
    const int first = win.a, k = win.k, n = win.n;
    // a warp sums an unbroken part of the row
    const int per = ((V - 1) / (32 * kWarps) + 1) * 32, lo = min(V, warp * per), hi = min(V, lo + per);
    const float u_in = a.sample_u[s];
    const double u = u_in > 0.f ? fmin((double)u_in, 1.0) : 0.0;
    for (int attempt = 0; attempt < 2; ++attempt) {
        Sum sum;
        for (int t = lo + lane; t < hi; t += 32) {
            const float2 v = w(t);
            sum.add(v.x, v.y);
        }
        const double mine = warp_total(sum);
        __syncthreads();
        if (lane == 0) part[warp] = mine;
        __syncthreads();
        double total = 0.0;
        for (int i = 0; i < kWarps; ++i) total += part[i];
        if (total > 0.0) {
            double goal = u * total;
            double before = 0.0;
            int owner = -1, last = -1;
            for (int i = 0; i < kWarps && owner < 0; ++i) {
                if (part[i] > 0.0) last = i;
                if (before + part[i] > goal) owner = i;
                else before += part[i];
            }
            if (owner < 0) {        // u = 1: the last token of any weight
                owner = last;
                goal = total * 2.0;
                before = 0.0;
            }
            if (warp == owner) {
                int at = -1, positive = -1;
                for (int base = lo; base < hi && at < 0; base += 32) {
                    const int t = base + lane;
                    const float2 v = t < hi ? w(t) : make_float2(0.f, 0.f);
                    double c = (double)v.x + (double)v.y;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double d = __shfl_up_sync(0xffffffffu, c, o);
                        if (lane >= o) c += d;
                    }
                    const uint32_t some = __ballot_sync(0xffffffffu, v.x > 0.f);
                    const uint32_t over = __ballot_sync(0xffffffffu, v.x > 0.f && before + c > goal);
                    if (some) positive = base + 31 - __clz(some);
                    if (over) at = base + __ffs(over) - 1;
                    before += __shfl_sync(0xffffffffu, c, 31);
                }
                if (lane == 0) found = at < 0 ? positive : at;
            }
            break;
        }
        if (w.q == nullptr && w.without < 0) break;     // nothing in the target's row either
        w.q = nullptr;
        w.without = -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= k; i += kThreads)
        a.out_tokens[first + i] = i < n ? a.tokens[first + i + 1] : i == n ? found : -1;
    if (threadIdx.x == 0) {
        if (found < 0) flag(a.device_status, SSD_DEV_BAD_PROBS);
        a.out_accepted[s] = n;
        if (a.ring_count) a.ring_count[s] += n + 1;
    }
}

}  // namespace

cudaError_t launch_verify(const ssd_verify_params &p, cudaStream_t stream) {
    if (p.prob_dtype == SSD_F32) return enqueue(verify_kernel<float>, dim3((unsigned)p.num_seqs), kThreads, stream, p);
    return enqueue(verify_kernel<__nv_bfloat16>, dim3((unsigned)p.num_seqs), kThreads, stream, p);
}

}  // namespace ssd
