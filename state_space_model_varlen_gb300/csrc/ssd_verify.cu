// Verification of drafted tokens: the first draft of a window that does not stand,
// and the token in its place (or behind the last draft).
//
//   draft i stands while u_i q_i(d_i) < p_i(d_i)
//   w = max(p - q, 0) of the row where it stopped;  new = the lowest t with cum_t > u cum_V
//
// The sums decide which whole number comes out, so they are kept to about 45 bits:
// pairs of floats whose additions keep what rounding drops (Knuth's two-sum; for
// p - q with p > q Dekker's shorter form).  Doubles would take longer than the reads:
// two operations a clock and SM, 16 clocks for one of a warp.
//
// A cluster of CTAs takes a window: each looks for the row where the window stops,
// sums its part of it, and learns the others' sums through distributed shared
// memory; the warp in whose part the random number falls reads that part again
// (from L2).  Bound by HBM for many windows, one row of p and one of q where a draft
// fell; for few by the chain of dependent reads in front of the row.
#include "ssd_layer_internal.h"
#include "ssd_mixer_common.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kLaneRun = 32;

// s + c, s the rounded sum
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ void add(float v, float rest) {
        const float t = s + v, b = t - s;
        c += ((s - (t - b)) + (v - b)) + rest;
        s = t;
    }
    __device__ void add(const Sum &o) { add(o.s, o.c); }
    __device__ void subtract(const Sum &o) { add(-o.s, -o.c); }
    __device__ bool above(const Sum &o) const { return (s - o.s) + (c - o.c) > 0.f; }
};
__device__ __forceinline__ Sum times(const Sum &a, float f) {
    Sum r;
    r.s = a.s * f;
    r.c = fmaf(a.s, f, -r.s) + a.c * f;
    return r;
}
__device__ __forceinline__ Sum shuffled(const Sum &a, int lane) {
    Sum r;
    r.s = __shfl_sync(0xffffffffu, a.s, lane);
    r.c = __shfl_sync(0xffffffffu, a.c, lane);
    return r;
}
// of lanes 0 .. lane
__device__ __forceinline__ Sum scan(Sum a) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float s = __shfl_up_sync(0xffffffffu, a.s, o), c = __shfl_up_sync(0xffffffffu, a.c, o);
        if ((threadIdx.x & 31) >= o) a.add(s, c);
    }
    return a;
}
// what scan() gave the lane before
__device__ __forceinline__ Sum before_lane(const Sum &a) {
    Sum r;
    r.s = __shfl_up_sync(0xffffffffu, a.s, 1);
    r.c = __shfl_up_sync(0xffffffffu, a.c, 1);
    return threadIdx.x & 31 ? r : Sum();
}
// The first of n lanes at which `sums`, scanned, pass goal, and what they are before
// it; or (with goal out of the way, so that the last of any weight is found below)
// the last one with a sum, or -1.
__device__ __forceinline__ int owner_of(const Sum &mine, int n, Sum &goal, Sum &before) {
    const int lane = threadIdx.x & 31;
    Sum upto = scan(lane < n ? mine : Sum());
    const Sum base = before;
    upto.add(base);
    Sum ahead = before_lane(upto);
    if (lane == 0) ahead = base;
    const uint32_t some = __ballot_sync(0xffffffffu, lane < n && mine.s > 0.f);
    const uint32_t over = some & __ballot_sync(0xffffffffu, upto.above(goal));
    if (!over) goal.s = __int_as_float(0x7f7fffff);
    const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
    before = shuffled(ahead, at < 0 ? 0 : at);
    return at;
}

// Where w comes from: the target's row, less the draft's row or what was drafted.
template <typename T> struct Weights {
    const T *p, *q;
    int without;                // token whose weight is 0, or -1
    // w of token t with probabilities a and b as a rounded value and what its rounding dropped
    __device__ static float2 of(float a, float b, bool out) {
        const float d = a - b;
        // 0 < d finite: a > b; b < 0 or not finite does not come with probabilities
        return d > 0.f && d < __int_as_float(0x7f800000) && !out ? make_float2(d, (a - d) - b) : make_float2(0.f, 0.f);
    }
    __device__ float2 operator()(int t) const { return of(to_float(p[t]), q ? to_float(q[t]) : 0.f, t == without); }
    // adds the weights of tokens t .. t + N - 1
    template <int N> __device__ void add(Sum &sum, int t) const {
        const Pack<T, N> a = load_pack<T, N>(p + t);
        Pack<T, N> b{};
        if (q) b = load_pack<T, N>(q + t);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 v = of(to_float(a.v[i]), to_float(b.v[i]), t + i == without);
            sum.add(v.x, v.y);
        }
    }
};

template <typename T> struct Window {
    int first, k, n;            // first token; drafts; drafts that stand
    bool live;
    Weights<T> w;
};

__device__ __forceinline__ void flag(int32_t *status, int bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ Sum load_of(const float2 *mine, int rank) {
    uint32_t at;
    Sum v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.s), "=f"(v.c) : "r"(at) : "memory");
    return v;
}

// The window's metadata and where it stops; one warp.  `report`: sets status bits.
template <typename T> __device__ void find_stop(const ssd_verify_params &a, int s, bool report, Window<T> &win) {
    const int lane = threadIdx.x & 31, V = a.vocab;
    const T *const target = static_cast<const T *>(a.target_probs), *const draft = static_cast<const T *>(a.draft_probs);
    const int64_t first = a.cu_seqlens[s], end = a.cu_seqlens[s + 1];
    const int64_t k = end - first - 1, d0 = first - s;
    bool ok = true;
    if (first < 0 || end < first || end > a.total_tokens || (k > 0 && (d0 < 0 || d0 + k > a.num_drafts))) {
        if (report && lane == 0) flag(a.device_status, SSD_DEV_BAD_SEQLENS);
        ok = false;
    }
    ok = ok && k >= 0;
    int n = 0;
    for (int base = 0; ok && base < k; base += 32) {
        const int i = base + lane;
        bool stands = true, bad = false;
        if (i < k) {
            const float u = a.accept_u[d0 + i];
            const int tok = a.tokens[first + i + 1];
            bad = tok < 0 || tok >= V;
            if (!bad) {
                const double q = draft ? (double)to_float(draft[(d0 + i) * a.draft_stride + tok]) : 1.0;
                const double p = (double)to_float(target[(first + i) * a.target_stride + tok]);
                stands = (double)fminf(fmaxf(u, 0.f), 1.f) * q < p;
            }
        }
        const uint32_t stop = __ballot_sync(0xffffffffu, bad || !stands), wrong = __ballot_sync(0xffffffffu, bad);
        if (stop) {
            const int at = __ffs(stop) - 1;
            n = base + at;
            if (wrong >> at & 1) {
                if (report && lane == 0) flag(a.device_status, SSD_DEV_BAD_TOKEN);
                ok = false;
            }
            break;
        }
        n = (int)min((int64_t)base + 32, k);
    }
    if (lane == 0) {
        win.live = ok;
        win.first = (int)first;
        win.k = (int)k;
        win.n = n;
        if (ok) {
            win.w.p = target + (first + n) * a.target_stride;
            win.w.q = draft && n < k ? draft + (d0 + n) * a.draft_stride : nullptr;
            win.w.without = !draft && n < k ? a.tokens[first + n + 1] : -1;
        }
    }
}

// The token of [lo, hi) where the sum, `before` ahead of lo, passes goal, or else the
// last of any weight (-1 without one).  A lane takes kLaneRun tokens in a row.
template <typename T, int N> __device__ int search(const Weights<T> &w, int lo, int hi, Sum before, const Sum &goal) {
    const int lane = threadIdx.x & 31;
    int positive = -1;
    for (int base = lo; base < hi; base += 32 * kLaneRun) {
        const int from = min(hi, base + lane * kLaneRun), to = min(hi, from + kLaneRun);
        Sum mine;
        int t = from;
#pragma unroll 4
        for (; t + N <= to; t += N) w.template add<N>(mine, t);
        for (; t < to; ++t) w.template add<1>(mine, t);
        const Sum run = scan(mine);
        Sum upto = run;
        upto.add(before);
        const uint32_t some = __ballot_sync(0xffffffffu, mine.s > 0.f), over = some & __ballot_sync(0xffffffffu, upto.above(goal));
        const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
        const Sum ahead = before_lane(run);
        if (at >= 0) {          // the lane's tokens one after another; its last of any weight where nothing passes
            int found = -1;
            if (lane == at) {
                Sum left = goal, so_far;
                left.subtract(before);
                left.subtract(ahead);
                for (int i = from; i < to; ++i) {
                    const float2 v = w(i);
                    so_far.add(v.x, v.y);
                    if (v.x > 0.f) {
                        found = i;
                        if (over && so_far.above(left)) break;
                    }
                }
            }
            positive = __shfl_sync(0xffffffffu, found, at);
            if (over) return positive;
        }
        before.add(shuffled(run, 31));
    }
    return positive;
}

template <typename T> __global__ void __launch_bounds__(kThreads, 2) verify_kernel(const ssd_verify_params a, int split, int per) {
    __shared__ Window<T> win;
    __shared__ float2 part[2][kWarps], totals[2];       // of the first attempt and of the second
    constexpr int N = 16 / sizeof(T);
    await_previous();
    const int s = blockIdx.x / split, rank = blockIdx.x % split, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = a.vocab;
    if (warp == 0) find_stop(a, s, rank == 0, win);
    const float u_in = a.sample_u[s], u = u_in > 0.f ? fminf(u_in, 1.f) : 0.f;
    __syncthreads();
    if (!win.live) return;              // of all CTAs of the cluster
    Weights<T> w = win.w;
    const int first = win.first, k = win.k, n = win.n;
    // a warp sums an unbroken part of the row
    const int64_t begin = ((int64_t)rank * kWarps + warp) * per;
    const int lo = (int)min((int64_t)V, begin), hi = (int)min((int64_t)V, begin + per);
    for (int attempt = 0;; ++attempt) {
        const bool wide = ((reinterpret_cast<uintptr_t>(w.p) | reinterpret_cast<uintptr_t>(w.q)) & 15) == 0;
        Sum sum;
        int t = lo;
        if (wide) {
#pragma unroll 4
            for (int i = lo + lane * N; i + N <= hi; i += 32 * N) w.template add<N>(sum, i);
            t = hi - (hi - lo) % N;
        }
#pragma unroll 8
        for (int i = t + lane; i < hi; i += 32) w.template add<1>(sum, i);
        const Sum mine = scan(sum);
        if (lane == 31) part[attempt][warp] = make_float2(mine.s, mine.c);
        __syncthreads();
        // every warp for itself, all the same: the CTA's sum, the others', and where the goal lies
        Sum warps;
        if (lane < kWarps) {
            warps.s = part[attempt][lane].x;
            warps.c = part[attempt][lane].y;
        }
        Sum cta = shuffled(scan(warps), kWarps - 1);
        if (split > 1) {
            if (threadIdx.x == 0) totals[attempt] = make_float2(cta.s, cta.c);
            cluster_arrive();
            cluster_wait();
            cta = lane < split ? load_of(&totals[attempt], lane) : Sum();
        }
        const Sum total = shuffled(scan(lane < split ? cta : Sum()), split - 1);
        const bool last_try = attempt == 1 || (w.q == nullptr && w.without < 0);
        if (total.s > 0.f || last_try) {
            Sum goal = times(total, u), before;
            if (u == 1.f) goal.s = __int_as_float(0x7f7fffff);          // the last of any weight
            const int owner = max(0, owner_of(cta, split, goal, before));
            if (rank == owner) {
                const int by = max(0, owner_of(warps, kWarps, goal, before));
                if (warp == by) {
                    const int at = wide ? search<T, N>(w, lo, hi, before, goal) : search<T, 1>(w, lo, hi, before, goal);
                    for (int i = lane; i <= k; i += 32) a.out_tokens[first + i] = i < n ? a.tokens[first + i + 1] : i == n ? at : -1;
                    if (lane == 0) {
                        if (at < 0) flag(a.device_status, SSD_DEV_BAD_PROBS);
                        a.out_accepted[s] = n;
                        if (a.ring_count) a.ring_count[s] += n + 1;
                    }
                }
            }
            break;
        }
        w.q = nullptr;                  // nothing is left of p - q: the target's row
        w.without = -1;
    }
    if (split > 1) {                    // no CTA leaves while another reads its sums
        cluster_arrive();
        cluster_wait();
    }
}

template <typename T> cudaError_t launch(const ssd_verify_params &p, cudaStream_t stream) {
    // CTAs of a window: parts of at least 4,096 tokens, about four CTAs an SM in all
    int split = 1;
    while (split < 8 && p.vocab >= split * 2 * 4096 && (int64_t)p.num_seqs * split * 2 <= 152 * 4) split *= 2;
    const int warps = split * kWarps;
    const int per = (int)((((int64_t)p.vocab - 1) / warps / 128 + 1) * 128);
    if ((int64_t)p.num_seqs * split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)(p.num_seqs * split));
    config.blockDim = dim3(kThreads);
    config.stream = stream;
    config.attrs = attr;
    config.numAttrs = 2;
    return cudaLaunchKernelEx(&config, verify_kernel<T>, p, split, per);
}

}  // namespace

cudaError_t launch_verify(const ssd_verify_params &p, cudaStream_t stream) {
    return p.prob_dtype == SSD_F32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace ssd
