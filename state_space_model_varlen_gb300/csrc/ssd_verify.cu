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

constexpr int kLaneRun = 32;

// s + c, s the rounded sum
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ void add(float v, float rest) {
        const float t = s + v, b = t - s;
        c += ((s - (t - b)) + (v - b)) + rest;
        s = t;
    }
    __device__ void add(const Sum &o) { add(o.s, o.c); }
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
    static constexpr int N = 16 / sizeof(T);
    const T *p, *q;
    int without;                // token whose weight is 0, or -1
    // w of a token with probabilities a and b as a rounded value and what its rounding dropped
    __device__ static float2 of(float a, float b, bool out) {
        const float d = a - b;
        // 0 < d finite: a > b; b < 0 or not finite does not come with probabilities
        return d > 0.f && d < __int_as_float(0x7f800000) && !out ? make_float2(d, (a - d) - b) : make_float2(0.f, 0.f);
    }
    __device__ float2 operator()(int t) const { return of(to_float(p[t]), q ? to_float(q[t]) : 0.f, t == without); }
    // elements that p's row begins behind a 16-byte boundary, and whether q's begins like it
    __device__ int ahead() const { return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T)); }
    __device__ bool alike() const { return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0; }
    __device__ void add_one(Sum &sum, int t) const {
        const float2 v = (*this)(t);
        sum.add(v.x, v.y);
    }
    // adds tokens t .. t + N - 1, where p + t is a 16-byte boundary
    __device__ void add(Sum &sum, int t, bool alike) const {
        const Pack<T, N> a = load_pack<T, N>(p + t);
        Pack<T, N> b{};
        if (q) {
            if (alike) {
                b = load_pack<T, N>(q + t);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) b.v[i] = q[t + i];
            }
        }
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
// last of any weight (-1 without one).  A lane takes kLaneRun tokens in a row, which
// begin at a 16-byte boundary of p but for the row's first.
template <typename T> __device__ int search(const Weights<T> &w, int lo, int hi, Sum before, const Sum &goal) {
    constexpr int N = Weights<T>::N;
    const int lane = threadIdx.x & 31, shift = w.ahead();
    const bool alike = w.alike();
    int positive = -1;
    for (int base = (lo + shift) / N * N - shift; base < hi; base += 32 * kLaneRun) {
        const int run = base + lane * kLaneRun;
        Sum mine;
#pragma unroll 4
        for (int t = run; t < run + kLaneRun; t += N) {
            if (t >= lo && t + N <= hi) {
                w.add(mine, t, alike);
            } else {
                for (int i = max(t, lo); i < min(t + N, hi); ++i) w.add_one(mine, i);
            }
        }
        const Sum upto = scan(mine);
        Sum all = upto;
        all.add(before);
        const uint32_t some = __ballot_sync(0xffffffffu, mine.s > 0.f), over = some & __ballot_sync(0xffffffffu, all.above(goal));
        const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
        if (at >= 0) {          // that lane's tokens, one a lane
            const Sum ahead = shuffled(before_lane(upto), at);
            const int t = base + at * kLaneRun + lane;
            Sum one;
            if (t >= lo && t < hi) w.add_one(one, t);
            Sum sum = scan(one);
            sum.add(ahead);
            sum.add(before);
            const uint32_t any = __ballot_sync(0xffffffffu, one.s > 0.f);
            const uint32_t passed = any & __ballot_sync(0xffffffffu, sum.above(goal));
            positive = base + at * kLaneRun + (over && passed ? __ffs(passed) - 1 : 31 - __clz(any));
            if (over) return positive;
        }
        before.add(shuffled(upto, 31));
    }
    return positive;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_kernel(const ssd_verify_params a, int split, int per) {
    constexpr int kWarps = kThreads / 32, N = Weights<T>::N;
    __shared__ Window<T> win;
    __shared__ float2 part[2][kWarps], totals[2];       // of the first attempt and of the second
    await_previous();
    const int s = blockIdx.x / split, rank = blockIdx.x % split, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = a.vocab;
    if (warp == 0) find_stop(a, s, rank == 0, win);
    const float u_in = a.sample_u[s], u = u_in > 0.f ? fminf(u_in, 1.f) : 0.f;
    __syncthreads();
    if (!win.live) return;              // of all CTAs of the cluster
    Weights<T> w = win.w;
    const int first = win.first, k = win.k, n = win.n;
    // a warp sums an unbroken part of the row, from a 16-byte boundary of p on
    const int64_t begin = ((int64_t)rank * kWarps + warp) * per - w.ahead();
    const int lo = (int)min((int64_t)V, max((int64_t)0, begin)), hi = (int)max((int64_t)0, min((int64_t)V, begin + per));
    const int lo_whole = min(hi, lo > 0 ? lo : (N - w.ahead()) % N), hi_whole = lo_whole + (hi - lo_whole) / N * N;
    for (int attempt = 0;; ++attempt) {
        const bool alike = w.alike();
        Sum sum;
        if (lo + lane < lo_whole) w.add_one(sum, lo + lane);
#pragma unroll 4
        for (int t = lo_whole + lane * N; t < hi_whole; t += 32 * N) w.add(sum, t, alike);
        if (hi_whole + lane < hi) w.add_one(sum, hi_whole + lane);
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
                    const int at = search(w, lo, hi, before, goal);
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

template <typename T, int kThreads> cudaError_t launch(const ssd_verify_params &p, int split, cudaStream_t stream) {
    constexpr int N = Weights<T>::N;
    const int warps = split * (kThreads / 32);
    const int per = (int)((((int64_t)p.vocab + N - 2) / warps / 128 + 1) * 128);       // of a row that begins N - 1 behind a boundary
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
    return cudaLaunchKernelEx(&config, verify_kernel<T, kThreads>, p, split, per);
}

template <typename T> cudaError_t launch(const ssd_verify_params &p, cudaStream_t stream) {
    // Threads of a window: as many as let all windows run at once (1,024 an SM), a
    // token to 16 of a row at most, so that the chain of reads in front of the row is
    // waited for once; in eight CTAs rather than in large ones.
    if (p.num_seqs > (1 << 28)) return cudaErrorInvalidConfiguration;
    int64_t threads = 152 * 1024 / p.num_seqs;
    if (threads > p.vocab / 16) threads = p.vocab / 16;
    const int size = threads >= 8 * 512 ? 512 : threads >= 8 * 256 ? 256 : 128;
    int split = 1;
    while (split < 8 && split * 2 * size <= threads) split *= 2;
    return size == 512   ? launch<T, 512>(p, split, stream)
           : size == 256 ? launch<T, 256>(p, split, stream)
                         : launch<T, 128>(p, split, stream);
}

}  // namespace

cudaError_t launch_verify(const ssd_verify_params &p, cudaStream_t stream) {
    return p.prob_dtype == SSD_F32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace ssd
