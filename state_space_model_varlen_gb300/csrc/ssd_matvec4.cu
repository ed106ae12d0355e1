// Products of few rows with 4-bit weights.
//
//   out[r, o] = bias[o] + sum_k scale[o, g(k)] (code[o, k] - zero[o, g(k)]) x[r, k]
//
// Here the kernel for any sizes, and the plan of the one on the tensor cores
// (ssd_matvec4_mma.cuh), which takes all but groups of odd sizes or below 16 columns,
// activation scales that no block of 32 columns keeps to, and rows of more than 2^20 columns.
#include "ssd_matvec4_mma.cuh"

namespace ssd {
namespace {

template <int kType> __device__ __forceinline__ float stored_value(const void *p, int64_t i) {
    using T = typename Stored<kType>::T;
    float v;
    decode<kType, 1>(load_pack<T, 1>(static_cast<const T *>(p) + i), &v);
    return v;
}
// element i of an array of the types of x and scale
__device__ __forceinline__ float value(const void *p, int64_t i, int type) {
    switch (type) {
        case SSD_F32: return stored_value<SSD_F32>(p, i);
        case SSD_BF16: return stored_value<SSD_BF16>(p, i);
        case SSD_F16: return stored_value<SSD_F16>(p, i);
        case SSD_E4M3: return stored_value<SSD_E4M3>(p, i);
    }
    return stored_value<SSD_I8>(p, i);
}
__device__ __forceinline__ void put(void *p, int64_t i, int type, float v) {
    if (type == SSD_F32) static_cast<float *>(p)[i] = v;
    else static_cast<__nv_bfloat16 *>(p)[i] = from_float<__nv_bfloat16>(v);
}

// ---------------------------------------------------------------------------
// Any sizes: a warp takes kOuts rows of weights, its lanes words of eight codes,
// against eight rows of x that the CTA keeps in shared memory, 1,024 columns at a
// time.  A weight is (code - zero) scale in fp32.  Bound by its fp32 operations: 1 row of
// 4,096 to 18,560 outputs 104 us.
// ---------------------------------------------------------------------------
constexpr int kAnyWarps = 8, kOuts = 2, kAnyRows = 8, kAnyColumns = 1024, kAnyWords = kAnyColumns / 8;

__global__ void __launch_bounds__(32 * kAnyWarps) matvec4_any_kernel(const ssd_matvec4_params a) {
    __shared__ float4 xs[kAnyRows][2][kAnyWords];       // the halves of a word's columns apart: no bank conflicts
    await_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int K = a.in_features, groups = (K - 1) / a.group_size + 1, x_groups = a.x_scale ? (K - 1) / a.x_group + 1 : 0;
    const int64_t bytes = ((int64_t)K + 1) / 2;
    const int r0 = blockIdx.y * kAnyRows, o0 = (blockIdx.x * kAnyWarps + warp) * kOuts;
    const int rows = min(kAnyRows, a.rows - r0);
    const bool eights = a.group_size % 8 == 0;
    float acc[kOuts][kAnyRows] = {};
    for (int k0 = 0; k0 < K; k0 += kAnyColumns) {
        __syncthreads();
        for (int i = threadIdx.x; i < kAnyRows * kAnyColumns; i += 32 * kAnyWarps) {
            const int r = i / kAnyColumns, c = i % kAnyColumns;
            const int64_t k = (int64_t)k0 + c;
            float v = 0.f;
            if (r < rows && k < K) {
                v = value(a.x, (int64_t)(r0 + r) * a.x_stride + k, a.x_dtype);
                if (a.x_scale) v *= a.x_scale[(int64_t)(r0 + r) * x_groups + k / a.x_group];
            }
            reinterpret_cast<float *>(&xs[r][(c >> 2) & 1][c >> 3])[c & 3] = v;
        }
        __syncthreads();
        for (int w = lane; w < kAnyWords && k0 + 8 * w < K; w += 32) {
            const int k = k0 + 8 * w;
            float f[kOuts][8];
#pragma unroll
            for (int j = 0; j < kOuts; ++j) {
                const int o = min(o0 + j, a.out_features - 1);
                const uint8_t *src = a.weight + (int64_t)o * a.weight_stride + k / 2;
                uint32_t word = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (k / 2 + b < bytes) word |= (uint32_t)src[b] << (8 * b);
                const int64_t base = (int64_t)o * groups;
                float s = 0.f, z = 8.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (i == 0 || !eights) {
                        const int64_t g = base + min(k + i, K - 1) / a.group_size;
                        s = value(a.scale, g, a.scale_dtype);
                        if (a.zero) z = (float)a.zero[g];
                    }
                    f[j][i] = ((float)(word >> (4 * i) & 15u) - z) * s;
                }
            }
#pragma unroll
            for (int r = 0; r < kAnyRows; ++r) {
                if (r >= rows) break;
                const float4 lo = xs[r][0][w], hi = xs[r][1][w];
                const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int j = 0; j < kOuts; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + i < K) acc[j][r] = fmaf(f[j][i], v[i], acc[j][r]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kOuts; ++j)
#pragma unroll
        for (int r = 0; r < kAnyRows; ++r) {
            const float v = lanes_sum<32>(acc[j][r]);
            const int o = o0 + j;
            if (lane == 0 && r < rows && o < a.out_features)
                put(a.out, (int64_t)(r0 + r) * a.out_stride + o, a.out_dtype,
                    a.bias ? v + value(a.bias, o, a.out_dtype) : v);
        }
}

cudaError_t launch_any(ssd_matvec4_params p, cudaStream_t stream) {
    if (p.x_dtype <= SSD_BF16) p.x_scale = nullptr;
    const int per = kAnyWarps * kOuts;
    const dim3 grid((p.out_features - 1) / per + 1, (p.rows - 1) / kAnyRows + 1);
    if (grid.y > 65535) return cudaErrorInvalidConfiguration;
    return enqueue(matvec4_any_kernel, grid, 32 * kAnyWarps, stream, p);
}

// ---------------------------------------------------------------------------
// The plan of the tensor-core kernel; false where it does not take the call.
// ---------------------------------------------------------------------------
int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

bool make_plan(const ssd_matvec4_params &p, Matvec4Plan &q, int &cols, int &shared, bool &whole) {
    using namespace matvec4;
    const int K = p.in_features, parts = p.x_dtype == SSD_F32 ? 3 : 1;
    if (K > (1 << 20)) return false;
    q.p = p;
    if (p.x_dtype <= SSD_BF16) q.p.x_scale = nullptr;
    q.groups = p.group_size >= K ? 1 : (K - 1) / p.group_size + 1;
    q.x_groups = !q.p.x_scale || p.x_group >= K ? 1 : (K - 1) / p.x_group + 1;
    const bool unbroken = q.groups == 1 || p.group_size % 32 == 0;
    if (!unbroken) {
        // groups of their own blocks, from a whole byte on, that do not waste most of them
        if (p.group_size % 2 != 0 || p.group_size < 16) return false;
        q.padded = p.group_size;
        q.group_blocks = (p.group_size - 1) / 32 + 1;
        q.blocks = q.groups * q.group_blocks;
    } else {
        q.blocks = (K - 1) / 32 + 1;
        q.group_blocks = q.groups == 1 ? q.blocks : p.group_size / 32;
    }
    if (q.x_groups == 1) q.x_group_blocks = q.blocks;
    else if (unbroken && p.x_group % 32 == 0) q.x_group_blocks = p.x_group / 32;
    else if (!unbroken && p.x_group == p.group_size) q.x_group_blocks = q.group_blocks;
    else return false;
    q.steps = (q.blocks - 1) / 4 + 1;
    auto magic = [](int blocks) { return (uint32_t)((1ull << 32) / blocks + 1); };
    q.group_magic = magic(q.group_blocks);
    q.x_group_magic = magic(q.x_group_blocks);
    // blocks that share their scales wherever a step begins
    shared = gcd(4, gcd(q.groups == 1 ? 4 : q.group_blocks, q.x_groups == 1 ? 4 : q.x_group_blocks));
    whole = unbroken && K % 32 == 0 && p.weight_stride % 16 == 0 && aligned_to(p.weight, 16);
    cols = 1;
    while (cols < 4 && cols * 8 < (int64_t)p.rows * parts) cols *= 2;
    q.row_tile = cols * 8 / parts < p.rows ? cols * 8 / parts : p.rows;
    q.x_rows = q.row_tile * parts;
    if ((p.rows - 1) / q.row_tile + 1 > 65535) return false;

    const int per_step = 4 / shared, scales = chunk(cols, shared) * per_step;
    const int steps_of_chunk = chunk(cols, shared);
    int at = kWarps * stages(shared, whole) * 16 * mats(cols) * pitch(shared, whole);
    auto take = [&](int bytes) {
        const int off = at;
        at += (bytes + 127) / 128 * 128;
        return off;
    };
    q.off_x = take(2 * q.x_rows * x_pitch(cols, shared));
    q.off_scale = take(2 * scales * scale_line(cols) * 4);
    q.off_zero = take(p.zero ? 2 * scales * scale_line(cols) * 4 : 0);
    q.off_xs = take(q.x_groups > 1 ? 2 * scales * cols * 8 * 4 : 0);
    q.smem = at;
    const int sums = (outs(cols) + 16) * q.x_rows * 4;
    if (q.smem < sums) q.smem = sums;
    if (q.smem > kSmemLimit) return false;

    // The split and the ways whose waves of CTAs take the least, in clocks.  A step is
    // about so many instructions of a warp; eight warps of an SM take a step in four
    // times as many clocks, 16 in seven; a chunk's x and scales take 800, a CTA begins
    // and ends in 5,000, in a cluster 7,000 (measured).
    const int fit = kSmemLimit / (q.smem + 1024), resident = fit < 1 ? 1 : fit < kCtas ? fit : kCtas;
    const int passes = (p.rows - 1) / q.row_tile + 1;
    const int work = 250 + 16 * cols + per_step * (20 + 12 * cols);
    const int chunks = (q.steps - 1) / steps_of_chunk + 1;
    double least = 0.0;
    for (int ways = 1; ways <= steps_of_chunk; ways *= 2) {
        const int outs_now = outs(cols) / ways, tiles = (p.out_features - 1) / outs_now + 1;
        for (int split = 1; split <= 8 && split <= chunks; split *= 2) {
            const int mine = (chunks - 1) / split + 1;
            const double all = (double)passes * tiles * split, rounds = all / (152 * resident), whole_rounds = (double)(int64_t)rounds;
            const double waves = whole_rounds < rounds ? whole_rounds + 1 : whole_rounds;
            const double cost = waves * ((split > 1 ? 7000 : 5000) + 800 * mine + mine * (steps_of_chunk / ways) * (double)work * (all <= 152 || resident == 1 ? 4 : 7));
            if (q.split == 0 || cost < least) {
                least = cost;
                q.split = split;
                q.ways = ways;
                q.tiles = tiles;
            }
        }
    }
    return true;
}

}  // namespace

cudaError_t launch_matvec4(const ssd_matvec4_params &p, cudaStream_t stream) {
    Matvec4Plan q = {};
    int cols, shared;
    bool whole;
    if (!make_plan(p, q, cols, shared, whole)) return launch_any(p, stream);
    return cols == 1   ? launch_matvec4_cols1(q, shared, whole, stream)
           : cols == 2 ? launch_matvec4_cols2(q, shared, whole, stream)
                       : launch_matvec4_cols4(q, shared, whole, stream);
}

}  // namespace ssd
