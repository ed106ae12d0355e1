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
// memory.  Lanes leave the sums of their blocks of tokens in shared memory, so that
// the warp in whose part the random number falls reads one block again (from L2).
//
// Bound by HBM for many windows, one row of p and one of q where a draft fell; for few
// by a chain of dependent reads (lengths, tokens, their probabilities, the row, the
// block again) and two cluster barriers.  Measured: one window of three tokens, 2^17
// tokens in fp32, 9.5 us (2.7 until the row is known, 3.5 for the row, 3 from there on);
// 128 windows 24.8 us, 4.1 TB/s (floor 15); 37 windows of one to nine tokens, 50,277 in
// bf16 (rows at every alignment) 9.5 us; 256 windows, whose sums cover two blocks each,
// all drafts rejected, 42.9 us (floor 39.6).  Before: one CTA a window 76 and 172 us, sums
// in doubles 19 and 68, the whole part read again 10 and 40, every number looked at
// for itself 9.4 and 28.
#include "ssd_layer_internal.h"
#include "ssd_mixer_common.cuh"

namespace ssd {
namespace {

constexpr int kSnaps = 8;        // blocks of a warp's part whose sums are left
// 16-byte vectors of a lane in a block, of n values each: 16 tokens, and 32 in a large
// CTA, whose part of a row of 2^17 is then one block, all of it asked for at once
constexpr int vectors(int threads, int n) { return (threads == 512 ? 32 : 16) / n; }

// s + c, s the rounded sum
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ void add(float v, float rest) {
        const float t = s + v, b = t - s;
        c += ((s - (t - b)) + (v - b)) + rest;
        s = t;
    }
    __device__ void add(float v) {
        const float t = s + v, b = t - s;
        c += (s - (t - b)) + (v - b);
        s = t;
    }
    __device__ void add(const Sum &o) { add(o.s, o.c); }
    // unit times this is above o; unit is a power of two
    __device__ bool above(const Sum &o, float unit) const { return fmaf(s, unit, -o.s) + fmaf(c, unit, -o.c) > 0.f; }
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
// of lanes 0 .. lane, over the first kLanes
template <int kLanes = 32> __device__ __forceinline__ Sum scan(Sum a) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
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
// The first of n lanes at which the sums `mine`, which are `upto` added up, pass goal
// from `before` on, and what they are before it; or (with goal out of the way, so that
// the last of any weight is found below) the last one with a sum, or -1.  `passed`: which
// of the two; goal does not tell, as it may be out of the way already.  goal is in
// 1 / unit, the sums are not.
__device__ __forceinline__ int owner_of(const Sum &mine, Sum upto, int n, Sum &goal, float unit, Sum &before, bool &passed) {
    const int lane = threadIdx.x & 31;
    Sum ahead = before_lane(upto);
    upto.add(before);
    ahead.add(before);
    const uint32_t some = __ballot_sync(0xffffffffu, lane < n && mine.s > 0.f);
    const uint32_t over = some & __ballot_sync(0xffffffffu, upto.above(goal, unit));
    passed = over != 0;
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
    // elements that p's row begins behind a 16-byte boundary, and whether q's begins like it
    __device__ int ahead() const { return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T)); }
    __device__ bool alike() const { return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0; }
    // w of tokens t .. t + N - 1, of which those in [lo, hi) count; p + t is a 16-byte boundary
    struct Vector {
        Pack<T, N> a, b;
        bool live;
    };
    __device__ Vector load(int t, int lo, int hi, bool alike) const {
        Vector v{};
        v.live = t < hi && t + N > lo;
        if (t >= lo && t + N <= hi) {
            v.a = load_pack<T, N>(p + t);
            if (q) {
                if (alike) {
                    v.b = load_pack<T, N>(q + t);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) v.b.v[i] = q[t + i];
                }
            }
        } else if (v.live) {        // the row's ends
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (t + i >= lo && t + i < hi) {
                    v.a.v[i] = p[t + i];
                    if (q) v.b.v[i] = q[t + i];
                }
        }
        return v;
    }
    // Adds them, fast where they are finite, which is seen from the sum; else one by one.
    __device__ void add(Sum &sum, const Vector &v, int t, int lo, int hi) const {
        if (!v.live) return;
        Sum now = sum;
        if (q) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float a = to_float(v.a.v[i]), b = to_float(v.b.v[i]), d = a - b;
                now.add(fmaxf(d, 0.f), d > 0.f ? (a - d) - b : 0.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) now.add(fmaxf(to_float(v.a.v[i]), 0.f));
        }
        if (!(now.s < __int_as_float(0x7f800000)) || (unsigned)(without - t) < (unsigned)N) now = careful(*this, sum, t, lo, hi);
        sum = now;
    }
    static __device__ __noinline__ Sum careful(const Weights w, Sum sum, int t, int lo, int hi) {
#pragma unroll 1
        for (int i = max(t, lo); i < min(t + N, hi); ++i) {
            const float2 f = of(to_float(w.p[i]), w.q ? to_float(w.q[i]) : 0.f, i == w.without);
            sum.add(f.x, f.y);
        }
        return sum;
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

// The token of a run of blocks of [lo, hi), the first at `base`, where the sum, `before`
// ahead of them, passes goal, or else the last of any weight.  One warp, whose lanes
// take unbroken runs of tokens.
template <typename T, int kVectors>
__device__ int search(const Weights<T> &w, int base, int blocks, int lo, int hi, Sum before, const Sum &goal, float unit, bool alike) {
    constexpr int N = Weights<T>::N, kRun = N * kVectors;
    const int lane = threadIdx.x & 31;
    int last = -1;
    for (int j = 0; j < blocks && base < hi; ++j, base += 32 * kRun) {
        typename Weights<T>::Vector v[kVectors];
        Sum mine;
#pragma unroll
        for (int i = 0; i < kVectors; ++i) v[i] = w.load(base + lane * kRun + i * N, lo, hi, alike);
#pragma unroll
        for (int i = 0; i < kVectors; ++i) w.add(mine, v[i], base + lane * kRun + i * N, lo, hi);
        const Sum upto = scan(mine);
        Sum limit = goal, ahead = before;
        bool here, there;               // the goal is in this run, or behind all that there is of this block
        const int at = owner_of(mine, upto, 32, limit, unit, ahead, here);
        if (at >= 0) {                  // that run's tokens, one a lane
            const int t = base + at * kRun + lane;
            Sum one;
            if (lane < kRun && t >= lo && t < hi) {
                const float2 f = Weights<T>::of(to_float(w.p[t]), w.q ? to_float(w.q[t]) : 0.f, t == w.without);
                one.add(f.x, f.y);
            }
            last = base + at * kRun + owner_of(one, scan<kRun>(one), kRun, limit, unit, ahead, there);
            if (here) return last;
        }
        before.add(shuffled(upto, 31));
    }
    return last;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 1 : 1024 / kThreads) verify_kernel(const ssd_verify_params a, int split, int per) {
    constexpr int kWarps = kThreads / 32, N = Weights<T>::N, kVectors = vectors(kThreads, N), kBlock = 32 * N * kVectors;
    __shared__ Window<T> win;
    __shared__ float2 part[2][kWarps], totals[2];       // of the first attempt and of the second
    __shared__ float2 snaps[kSnaps][kThreads];
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
    const int base = lo > 0 ? lo : -w.ahead();
    const int runs = (per / kBlock - 1) / kSnaps + 1;           // blocks of a sum that is left
    for (int attempt = 0;; ++attempt) {
        const bool alike = w.alike();
        Sum sum;
        for (int i = 0; i < kSnaps; ++i) {
            Sum here;
            for (int j = 0; j < runs; ++j) {
                const int at = base + (i * runs + j) * kBlock + lane * N;
                if (at - lane * N >= hi) break;
                typename Weights<T>::Vector v[kVectors];
#pragma unroll
                for (int e = 0; e < kVectors; ++e) v[e] = w.load(at + e * 32 * N, lo, hi, alike);
#pragma unroll
                for (int e = 0; e < kVectors; ++e) w.add(here, v[e], at + e * 32 * N, lo, hi);
            }
            snaps[i][threadIdx.x] = make_float2(here.s, here.c);
            sum.add(here);
        }
        const Sum mine = scan(sum);
        if (lane == 31) part[attempt][warp] = make_float2(mine.s, mine.c);
        __syncthreads();
        // every warp for itself, all the same: the CTA's sum, the others', and where the goal lies
        Sum warps, ctas;
        if (lane < kWarps) {
            warps.s = part[attempt][lane].x;
            warps.c = part[attempt][lane].y;
        }
        const Sum warps_upto = scan<kWarps>(warps);
        ctas = shuffled(warps_upto, kWarps - 1);
        if (split > 1) {
            if (threadIdx.x == 0) totals[attempt] = make_float2(ctas.s, ctas.c);
            cluster_arrive();
            cluster_wait();
            ctas = lane < split ? load_of(&totals[attempt], lane) : Sum();
        }
        const Sum ctas_upto = scan<8>(ctas);
        Sum total = shuffled(ctas_upto, split - 1);
        const bool last_try = attempt == 1 || (w.q == nullptr && w.without < 0);
        if (total.s > 0.f || last_try) {
            // u total is a fraction of fp32's smallest numbers where the total is small: there in 2^-80
            const float unit = total.s < 8.673617379884035e-19f ? 1.2089258196146292e24f : 1.f;         // 2^-60, 2^80
            total.s *= unit;
            total.c *= unit;
            Sum goal = times(total, u), before;
            if (u == 1.f) goal.s = __int_as_float(0x7f7fffff);          // the last of any weight
            bool passed;
            const int owner = max(0, owner_of(ctas, ctas_upto, split, goal, unit, before, passed));
            if (rank == owner) {
                const int by = max(0, owner_of(warps, warps_upto, kWarps, goal, unit, before, passed));
                if (warp == by) {
                    // the sums of the warp's blocks: four lanes add one's 32, then the block of the goal
                    __syncwarp();
                    Sum run;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 v = snaps[lane >> 2][warp * 32 + (lane & 3) * 8 + i];
                        run.add(v.x, v.y);
                    }
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) run.add(__shfl_xor_sync(0xffffffffu, run.s, o), __shfl_xor_sync(0xffffffffu, run.c, o));
                    if (lane & 3) run = Sum();
                    const int from = max(0, owner_of(run, scan(run), 32, goal, unit, before, passed)) >> 2;
                    // a sum that fp32 does not hold is infinite, and says nothing of where the goal lies
                    const int at = total.s < __int_as_float(0x7f800000)
                                       ? search<T, kVectors>(w, base + from * runs * kBlock, runs, lo, hi, before, goal, unit, alike)
                                       : -1;
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
    constexpr int N = Weights<T>::N, kBlock = 32 * N * vectors(kThreads, N);
    const int warps = split * (kThreads / 32);
    // tokens that a row may begin behind a 16-byte boundary
    const int slack = aligned_to(p.target_probs, 16) && p.target_stride % N == 0 ? 0 : N - 1;
    const int per = (int)((((int64_t)p.vocab + slack - 1) / warps / kBlock + 1) * kBlock);
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
    config.numAttrs = split > 1 ? 2 : 1;
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
