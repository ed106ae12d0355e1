// Products of few rows with 4-bit weights on the tensor cores, for rows of weights
// in whole 16 bytes and groups of a multiple of 32 columns.
//
// A tile is 16 outputs, or 32 for few columns; a warp multiplies it by 128 columns at a step
// (mma.m16n8k16, weights as the 16 rows, rows of x as the columns).  code - zero is
// an integer below 2^4 and exact in bf16, as are 8-bit activations; fp32 activations
// become three bf16 parts of eight bits each, which together are exact.  Sums within
// a group are the instruction's fp32 sums, the groups' scales are applied to them
// in fp32.
//
// Bound by HBM: codes stream through a ring of asynchronous copies of each warp's
// own, kStages steps deep; x is in shared memory for good.  The columns of a tile
// are split over the warps of a CTA, and over a cluster of CTAs where there are few
// tiles; the parts are added in a fixed order.
#include "ssd_layer_internal.h"
#include "ssd_mixer_common.cuh"

namespace ssd {
namespace {

constexpr int kStages = 3, kMaxWarps = 8, kStep = 128;
constexpr int kSmemLimit = 227 * 1024;

struct Plan {
    ssd_matvec4_params p;
    int row_tile;               // rows of x of a pass
    int split;                  // CTAs of a cluster, which share a tile's columns
    int warps;
    int tiles, clusters;
    int steps;                  // of a row: ceil(K / 128)
    int per_warp;               // steps of a warp for one tile
    int groups, x_groups;       // of a row
    int group_blocks, x_group_blocks;   // 32-column blocks of a group
    uint32_t group_magic, x_group_magic;        // floor(2^32 / blocks) + 1
    int slice_x_groups;         // most x groups that a CTA's columns meet
    int x_stride;               // bytes of a row of x in shared memory
    int scale_slots;            // tiles whose scales are held
    int scale_bytes, zero_bytes;        // of a tile
    int off_x, off_xs, off_scale, off_zero, off_part, off_own, smem;
};

__device__ __forceinline__ int group_of(int block, int blocks, uint32_t magic) {
    return blocks == 1 ? block : (int)__umulhi((uint32_t)block, magic);
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// v in a register, which the compiler does not load or compute again at each use.
__device__ __forceinline__ int kept(int v) {
    int r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Codes i and i + 4 of a word (at bits 4 i and 4 i + 16) less their zero, as bf16:
// the code as the low bits of 128's mantissa, minus 128 + zero.  Exact.
__device__ __forceinline__ uint32_t codes2(uint32_t word, int i, uint32_t base, uint32_t zero) {
    uint32_t v, r;              // and, or as one operation (the compiler makes two)
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(word >> (4 * i)), "n"(0x000f000f), "r"(base));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero));
    return r;
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// eight consecutive values of a row of x
__device__ __forceinline__ void load8(float (&v)[8], const ssd_matvec4_params &p, int64_t at, int live, bool wide) {
    if (wide && live == 8) {
        if (p.x_dtype == SSD_F32) {
            const auto a = load_pack<float, 8>(static_cast<const float *>(p.x) + at);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = a.v[i];
        } else if (p.x_dtype == SSD_BF16) {
            decode<SSD_BF16, 8>(load_pack<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16 *>(p.x) + at), v);
        } else {
            const auto a = load_pack<uint8_t, 8>(static_cast<const uint8_t *>(p.x) + at);
            if (p.x_dtype == SSD_E4M3) decode<SSD_E4M3, 8>(a, v);
            else decode<SSD_I8, 8>(a, v);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = 0.f;
        if (i >= live) continue;
        const int64_t e = at + i;
        if (p.x_dtype == SSD_F32) v[i] = static_cast<const float *>(p.x)[e];
        else if (p.x_dtype == SSD_BF16) v[i] = to_float(static_cast<const __nv_bfloat16 *>(p.x)[e]);
        else if (p.x_dtype == SSD_E4M3) decode<SSD_E4M3, 1>(load_pack<uint8_t, 1>(static_cast<const uint8_t *>(p.x) + e), v + i);
        else decode<SSD_I8, 1>(load_pack<uint8_t, 1>(static_cast<const uint8_t *>(p.x) + e), v + i);
    }
}

// The block of `bytes` (a multiple of 16) at src into shared memory, zeros behind the
// first `live`: asynchronously in 16 bytes where src is aligned, else at once.
__device__ __noinline__ void copy_ragged(uint8_t *dst, const uint8_t *src, int bytes, int live) {
    for (int i = threadIdx.x; i < bytes; i += blockDim.x) dst[i] = i < live ? src[i] : 0;
}
__device__ __forceinline__ void copy_block(uint8_t *dst, const uint8_t *src, int bytes, int live, int thread) {
    if (live == bytes && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll 1
        for (int i = thread * 16; i < bytes; i += blockDim.x * 16) copy_async<16>(dst + i, src + i, true);
    } else {
        copy_ragged(dst, src, bytes, live);
    }
}

// kCols: eights of columns (rows of x, or their parts) of a pass.  kBlocks: 32-column
// blocks that certainly share their scales (1, 2, or 4: a step).
constexpr int mats(int cols) { return cols <= 2 ? 2 : 1; }         // sixteens of outputs of a tile
constexpr int ctas(int cols) { return cols <= 4 ? 2 : 1; }
constexpr int pitch(int blocks) { return blocks == 4 ? 64 : 80; }   // bytes of a row of a stage: no bank conflicts

template <int kCols, int kBlocks, bool kX8, bool kZero>
__global__ void __launch_bounds__(32 * kMaxWarps, ctas(kCols)) matvec4_mma_kernel(const __grid_constant__ Plan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kMats = mats(kCols), kTile = 16 * kMats, kPitch = pitch(kBlocks), kWide = kCols * 8;
    const ssd_matvec4_params &p = plan.p;
    const int thread = kept(threadIdx.x), lane = thread & 31, g = lane >> 2, t = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, thread >> 5, 0);          // known to be the same in all lanes
    const uint32_t base = (uint32_t)kept(0x43004300);                  // 128 in bf16, twice
    const int scale_type = kept(p.scale_dtype);
    const int rank = blockIdx.x % plan.split, cluster = blockIdx.x / plan.split;
    const int r0 = blockIdx.y * plan.row_tile, rows = min(plan.row_tile, p.rows - r0);
    const int parts = p.x_dtype == SSD_F32 ? 3 : 1, cols = rows * parts, wide = (cols + 1) & ~1;
    const int step0 = (int)((int64_t)plan.steps * rank / plan.split), step1 = (int)((int64_t)plan.steps * (rank + 1) / plan.split);
    const int K = p.in_features, row_bytes = kept(K / 2), warps = kept(plan.warps), per_warp = kept(plan.per_warp);
    uint8_t *const ring = smem + warp * (kStages * kTile * kPitch);
    uint8_t *const xs = smem + plan.off_x;
    float *const xsc = reinterpret_cast<float *>(smem + plan.off_xs);
    float *const part = reinterpret_cast<float *>(smem + plan.off_part);
    float *const own = reinterpret_cast<float *>(smem + plan.off_own);
    const int my_tiles = (plan.tiles - cluster + plan.clusters - 1) / plan.clusters;
        await_previous();

    // scales and zeros of the next tile whose codes are asked for
    const int64_t tile_scales = (int64_t)plan.clusters * plan.scale_bytes, tile_zeros = (int64_t)plan.clusters * plan.zero_bytes;
    const uint8_t *scale_src = static_cast<const uint8_t *>(p.scale) + (int64_t)cluster * plan.scale_bytes;
    const uint8_t *zero_src = kZero ? p.zero + (int64_t)cluster * plan.zero_bytes : nullptr;
    const int whole_tiles = p.out_features / kTile, whole_steps = K / kStep;
    auto copy_scales = [&](int at, int slot) {          // of the tile that is number `at` of all
        const int live = at < whole_tiles ? kTile : p.out_features - at * kTile;
        copy_block(smem + plan.off_scale + slot * plan.scale_bytes, scale_src, plan.scale_bytes,
                   live * (plan.scale_bytes / kTile), thread);
        scale_src += tile_scales;
        if (kZero) {
            copy_block(smem + plan.off_zero + slot * plan.zero_bytes, zero_src, plan.zero_bytes, live * plan.groups, thread);
            zero_src += tile_zeros;
        }
    };
    // The next step's codes, and with a tile's last step the scales of the next tile,
    // which are then complete for all when this tile has been added up.
    int to_tile = 0, to_step = step0 + warp, to_j = 0, to_stage = 0, to_slot = 0;
    const uint8_t *src[2 * kMats];                      // of the lane's 16 bytes of its rows
    auto point = [&]() {
#pragma unroll
        for (int h = 0; h < 2 * kMats; ++h) {
            const int64_t o = min((int64_t)(cluster + to_tile * plan.clusters) * kTile + g + 8 * h, (int64_t)p.out_features - 1);
            src[h] = p.weight + o * p.weight_stride + (t * 16 < row_bytes ? t * 16 : 0);
        }
    };
    point();
    uint8_t *const to = ring + g * kPitch + t * 16;
    const int64_t jump = (int64_t)plan.clusters * kTile * p.weight_stride;
    auto issue = [&]() {
        if (to_tile < my_tiles) {
            if (to_step < step1) {
                const int byte = to_step * (kStep / 2);
                uint8_t *const dst = to + to_stage * (kTile * kPitch);
                if (to_step < whole_steps) {
#pragma unroll
                    for (int h = 0; h < 2 * kMats; ++h) copy_async<16>(dst + 8 * h * kPitch, src[h] + byte, true);
                } else {                                // the columns of the last step that are there
                    const bool live = byte + t * 16 < row_bytes;
#pragma unroll
                    for (int h = 0; h < 2 * kMats; ++h) copy_async<16>(dst + 8 * h * kPitch, src[h] + (live ? byte : 0), live);
                }
            }
            to_step += warps;
            if (++to_j == per_warp) {
                to_j = 0;
                to_step = step0 + warp;
                if (++to_tile < my_tiles) {
                    const int at = cluster + to_tile * plan.clusters;
                    to_slot = to_slot + 1 == plan.scale_slots ? 0 : to_slot + 1;
                    copy_scales(at, to_slot);
                    if (at < whole_tiles) {
#pragma unroll
                        for (int h = 0; h < 2 * kMats; ++h) src[h] += jump;
                    } else {
                        point();
                    }
                }
            }
        }
        to_stage = to_stage + 1 == kStages ? 0 : to_stage + 1;
        commit_async();
    };

    if (my_tiles > 0) copy_scales(cluster, 0);
#pragma unroll 1
    for (int q = 0; q < kStages - 1; ++q) issue();

    // x of the CTA's columns as bf16, in chunks of eight: values i and i + 4 side by
    // side, as the codes of a word come; within a step the chunk that quad lane t reads
    // with its j-th word at 4 j + t
    {
        const int chunks = (step1 - step0) * 16;
        const int size = p.x_dtype == SSD_F32 ? 16 : p.x_dtype == SSD_BF16 ? 16 : 8;
        const int elem = p.x_dtype == SSD_F32 ? 4 : p.x_dtype == SSD_BF16 ? 2 : 1;
        const bool wide = (reinterpret_cast<uintptr_t>(p.x) % size) == 0 && (p.x_stride * elem) % size == 0;
        for (int i = threadIdx.x; i < rows * chunks; i += blockDim.x) {
            const int r = i / chunks, c = i - r * chunks;
            const int64_t k = (int64_t)step0 * kStep + c * 8;
            float v[8];
            load8(v, p, (r0 + r) * p.x_stride + k, (int)max((int64_t)0, min((int64_t)8, K - k)), wide);
            const int at = kBlocks == 4 ? (c & ~15) | (c & 3) << 2 | (c >> 2 & 3) : c;
            for (int part = 0; part < parts; ++part) {
                uint32_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u[j] = __float_as_uint(v[j]);
                    if (v[j] != v[j]) u[j] = 0x7fc00000u;
                    const float cut = __uint_as_float(u[j] & 0xffff0000u);
                    v[j] = fabsf(cut) < __int_as_float(0x7f800000) ? v[j] - cut : 0.f;
                }
                const uint4 w = make_uint4(__byte_perm(u[0], u[4], 0x7632), __byte_perm(u[1], u[5], 0x7632),
                                           __byte_perm(u[2], u[6], 0x7632), __byte_perm(u[3], u[7], 0x7632));
                *reinterpret_cast<uint4 *>(xs + (part * rows + r) * plan.x_stride + at * 16) = w;
            }
        }
        if constexpr (kX8) {
            const int first = group_of(step0 * 4, plan.x_group_blocks, plan.x_group_magic);
            for (int i = threadIdx.x; i < plan.slice_x_groups * kWide; i += blockDim.x) {
                const int r = i % kWide, x_group = first + i / kWide;
                xsc[i] = r < rows && x_group < plan.x_groups ? p.x_scale[(int64_t)(r0 + r) * plan.x_groups + x_group] : 0.f;
            }
        }
    }
    wait_async<kStages - 2>();
    __syncthreads();

    const int first_x_group = kX8 ? group_of(step0 * 4, plan.x_group_blocks, plan.x_group_magic) : 0;
    int row_at[2 * kMats];                              // of the lane's rows in a tile's scales
#pragma unroll
    for (int h = 0; h < 2 * kMats; ++h) row_at[h] = (g + 8 * h) * plan.groups;
    // A column that is not there is computed from the last one and not looked at.
    int x_at[kCols];
#pragma unroll
    for (int n = 0; n < kCols; ++n) x_at[n] = min(n * 8 + g, cols - 1) * plan.x_stride + t * 16;
    float sum[kMats][kCols][4];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[m][n][i] = 0.f;
    int stage = 0, slot = 0;
    const uint32_t eight = (uint32_t)kept(0x43084308);  // 128 + 8
    for (int tile = 0; tile < my_tiles; ++tile) {
        const uint8_t *const scales = smem + plan.off_scale + slot * plan.scale_bytes;
        const uint8_t *const zeros = smem + plan.off_zero + slot * plan.zero_bytes;
        slot = slot + 1 == plan.scale_slots ? 0 : slot + 1;
        int step = step0 + warp;
#pragma unroll 1
        for (int j = 0; j < per_warp; ++j, step += warps) {
            wait_async<kStages - 2>();
            if constexpr (kBlocks < 4) __syncwarp();    // a lane reads what its neighbours copied
            issue();
            const uint8_t *const codes = ring + stage * (kTile * kPitch) + g * kPitch + (kBlocks == 4 ? t * 16 : t * 4);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            if (step >= step1) continue;
            const uint8_t *const x = xs + (step - step0) * (kStep * 2);
            uint32_t words[2 * kMats][4];
            if constexpr (kBlocks == 4) {
#pragma unroll
                for (int h = 0; h < 2 * kMats; ++h)
                    *reinterpret_cast<uint4 *>(words[h]) = *reinterpret_cast<const uint4 *>(codes + 8 * h * kPitch);
            }
#pragma unroll
            for (int f = 0; f < 4 / kBlocks; ++f) {
                const int block = step * 4 + f * kBlocks;
                if (kBlocks < 4 && block * 32 >= K) break;
                const int gi = group_of(block, plan.group_blocks, plan.group_magic);
                uint32_t zero[2 * kMats];               // 128 + zero, twice
#pragma unroll
                for (int h = 0; h < 2 * kMats; ++h)
                    zero[h] = kZero ? base + zeros[row_at[h] + gi] * 0x00010001u : eight;
                float acc[kMats][kCols][4];
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const int w = f * kBlocks + b;
                    uint32_t a0[kMats][4], a1[kMats][4];
#pragma unroll
                    for (int m = 0; m < kMats; ++m) {
                        uint32_t lo = words[2 * m][w], hi = words[2 * m + 1][w];
                        if constexpr (kBlocks < 4) {
                            lo = *reinterpret_cast<const uint32_t *>(codes + 16 * m * kPitch + w * 16);
                            hi = *reinterpret_cast<const uint32_t *>(codes + (16 * m + 8) * kPitch + w * 16);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a0[m][2 * i] = codes2(lo, i, base, zero[2 * m]);
                            a0[m][2 * i + 1] = codes2(hi, i, base, zero[2 * m + 1]);
                            a1[m][2 * i] = codes2(lo, i + 2, base, zero[2 * m]);
                            a1[m][2 * i + 1] = codes2(hi, i + 2, base, zero[2 * m + 1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kCols; ++n) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(x + x_at[n] + w * 64);
#pragma unroll
                        for (int m = 0; m < kMats; ++m) {
                            if (b == 0) mma_first(acc[m][n], a0[m], v.x, v.y);
                            else mma(acc[m][n], a0[m], v.x, v.y);
                            mma(acc[m][n], a1[m], v.z, v.w);
                        }
                    }
                }
                float scale[2 * kMats];
                if (scale_type == SSD_F32) {
#pragma unroll
                    for (int h = 0; h < 2 * kMats; ++h) scale[h] = reinterpret_cast<const float *>(scales)[row_at[h] + gi];
                } else {
#pragma unroll
                    for (int h = 0; h < 2 * kMats; ++h) {
                        const uint16_t v = reinterpret_cast<const uint16_t *>(scales)[row_at[h] + gi];
                        const float bf16 = __uint_as_float((uint32_t)v << 16), f16 = __half2float(__ushort_as_half(v));
                        scale[h] = scale_type == SSD_BF16 ? bf16 : f16;
                    }
                }
                const int xg = kX8 ? group_of(block, plan.x_group_blocks, plan.x_group_magic) - first_x_group : 0;
#pragma unroll
                for (int n = 0; n < kCols; ++n) {
                    if constexpr (kX8) {
                        const float2 s = *reinterpret_cast<const float2 *>(xsc + (xg * kCols + n) * 8 + 2 * t);
#pragma unroll
                        for (int m = 0; m < kMats; ++m) {
                            acc[m][n][0] *= s.x;
                            acc[m][n][1] *= s.y;
                            acc[m][n][2] *= s.x;
                            acc[m][n][3] *= s.y;
                        }
                    }
#pragma unroll
                    for (int m = 0; m < kMats; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[m][n][i] = fmaf(acc[m][n][i], scale[2 * m + i / 2], sum[m][n][i]);
                }
            }
        }
        // the tile's parts: of the warps, then of the cluster's CTAs.  Two buffers, so
        // that one barrier a tile is enough.
        const float *const all = part + (tile & 1) * warps * (kTile * wide);
        float *const mine = part + ((tile & 1) * warps + warp) * (kTile * wide);
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
                float *const at = mine + (16 * m + g) * wide + n * 8 + 2 * t;
                if (n * 8 + 2 * t < wide) {
                    *reinterpret_cast<float2 *>(at) = make_float2(sum[m][n][0], sum[m][n][1]);
                    *reinterpret_cast<float2 *>(at + 8 * wide) = make_float2(sum[m][n][2], sum[m][n][3]);
                }
                sum[m][n][0] = sum[m][n][1] = sum[m][n][2] = sum[m][n][3] = 0.f;
            }
        __syncthreads();
        const int o0 = (cluster + tile * plan.clusters) * kTile;
        auto finish = [&](int i, float v) {             // output i of the tile's rows x kTile
            const int r = i / kTile, o = o0 + i % kTile;
            if (o >= p.out_features) return;
            const int64_t at = (r0 + r) * p.out_stride + o;
            if (p.out_dtype == SSD_F32) {
                if (p.bias) v += static_cast<const float *>(p.bias)[o];
                static_cast<float *>(p.out)[at] = v;
            } else {
                if (p.bias) v += to_float(static_cast<const __nv_bfloat16 *>(p.bias)[o]);
                static_cast<__nv_bfloat16 *>(p.out)[at] = from_float<__nv_bfloat16>(v);
            }
        };
        float *const own_now = own + (tile & 1) * (kTile * rows);
        for (int i = thread; i < rows * kTile; i += blockDim.x) {
            const float *at = all + i % kTile * wide + i / kTile;
            float v = 0.f;
            for (int w = 0; w < warps; ++w, at += kTile * wide) {
                v += at[0];
                if (parts == 3) v += at[rows] + at[2 * rows];
            }
            if (plan.split == 1) finish(i, v);
            else own_now[i] = v;
        }
        if (plan.split > 1) {
            cluster_barrier();
            const uint32_t local = (uint32_t)__cvta_generic_to_shared(own_now);
            for (int i = rank * blockDim.x + thread; i < rows * kTile; i += plan.split * blockDim.x) {
                float v = 0.f;
                for (int c = 0; c < plan.split; ++c) {
                    uint32_t at;
                    float f;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local + i * 4), "r"(c));
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(at) : "memory");
                    v += f;
                }
                finish(i, v);
            }
        }
    }
    // no CTA leaves while another reads its part
    if (plan.split > 1) cluster_barrier();
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }
int up(int v, int to) { return (v + to - 1) / to * to; }

// Shared memory of a plan whose split, warps and rows are set.
void lay_out(Plan &q, int col_tiles, int blocks) {
    const int kTile = 16 * mats(col_tiles);
    const int parts = q.p.x_dtype == SSD_F32 ? 3 : 1, slice = (q.steps - 1) / q.split + 1;
    q.per_warp = (slice - 1) / q.warps + 1;
    q.x_stride = up(slice * kStep * 2, 128) + 64;       // two rows of x beside one another in the banks
    q.scale_slots = (kStages - 1) / q.per_warp + 2;
    const int size = q.p.scale_dtype == SSD_F32 ? 4 : 2;
    q.scale_bytes = kTile * q.groups * size;
    q.zero_bytes = q.p.zero ? kTile * q.groups : 0;
    q.slice_x_groups = q.p.x_scale ? slice * 4 / q.x_group_blocks + 2 : 0;
    int at = q.warps * kStages * kTile * pitch(blocks);
    auto take = [&](int bytes) {
        const int off = at;
        at += up(bytes, 128);
        return off;
    };
    q.off_x = take(q.row_tile * parts * q.x_stride);
    q.off_xs = take(q.slice_x_groups * col_tiles * 8 * 4);
    q.off_scale = take(q.scale_slots * q.scale_bytes);
    q.off_zero = take(q.scale_slots * q.zero_bytes);
    q.off_part = take(2 * q.warps * kTile * up(q.row_tile * parts, 2) * 4);
    q.off_own = take(q.split > 1 ? 2 * kTile * q.row_tile * 4 : 0);
    q.smem = at;
}

template <int kCols, int kBlocks, bool kX8, bool kZero> cudaError_t run(const Plan &q, cudaStream_t stream) {
    auto kernel = matvec4_mma_kernel<kCols, kBlocks, kX8, kZero>;
    // the most that any plan takes, so that one call of a process and device is enough
    static unsigned long long set = 0;          // bit d: device d (the first 64)
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= 64 || !(__atomic_load_n(&set, __ATOMIC_ACQUIRE) >> device & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
        if (device < 64) __atomic_fetch_or(&set, 1ull << device, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)q.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)(q.clusters * q.split), (unsigned)((q.p.rows - 1) / q.row_tile + 1));
    config.blockDim = dim3((unsigned)(32 * q.warps));
    config.dynamicSmemBytes = (size_t)q.smem;
    config.stream = stream;
    config.attrs = attr;
    config.numAttrs = 2;
    return cudaLaunchKernelEx(&config, kernel, q);
}

template <int kCols, int kBlocks> cudaError_t run(const Plan &q, cudaStream_t stream) {
    if (q.p.zero) return q.p.x_scale ? run<kCols, kBlocks, true, true>(q, stream) : run<kCols, kBlocks, false, true>(q, stream);
    return q.p.x_scale ? run<kCols, kBlocks, true, false>(q, stream) : run<kCols, kBlocks, false, false>(q, stream);
}

template <int kCols> cudaError_t run(const Plan &q, int blocks, cudaStream_t stream) {
    return blocks == 4   ? run<kCols, 4>(q, stream)
           : blocks == 2 ? run<kCols, 2>(q, stream)
                         : run<kCols, 1>(q, stream);
}

}  // namespace

bool launch_matvec4_mma(const ssd_matvec4_params &p, cudaStream_t stream, cudaError_t *error) {
    auto whole = [&](int group) { return group % 32 == 0 || group >= p.in_features; };
    if (p.in_features % 32 != 0 || p.in_features > (1 << 20) || p.weight_stride % 16 != 0 || !aligned_to(p.weight, 16) ||
        !whole(p.group_size) || (p.x_dtype > SSD_BF16 && !whole(p.x_group)))
        return false;
    Plan q = {};
    q.p = p;
    if (p.x_dtype <= SSD_BF16) q.p.x_scale = nullptr;
    const int K = p.in_features, parts = p.x_dtype == SSD_F32 ? 3 : 1;
    auto blocks_of = [&](int group) { return group >= K ? K / 32 : group / 32; };
    q.groups = p.group_size >= K ? 1 : (K - 1) / p.group_size + 1;
    q.group_blocks = blocks_of(p.group_size);
    q.x_groups = !q.p.x_scale || p.x_group >= K ? 1 : (K - 1) / p.x_group + 1;
    q.x_group_blocks = q.p.x_scale ? blocks_of(p.x_group) : 1;
    auto magic = [](int blocks) { return (uint32_t)((1ull << 32) / blocks + 1); };
    q.group_magic = magic(q.group_blocks);
    q.x_group_magic = magic(q.x_group_blocks);
    // blocks that share their scales wherever a step begins
    const int wb = q.groups == 1 ? 4 : q.group_blocks, xb = q.x_groups == 1 ? 4 : q.x_group_blocks;
    const int blocks = gcd(4, gcd(wb, xb));
    q.steps = (K - 1) / kStep + 1;
    int col_tiles = 1;
    while (col_tiles < 8 && col_tiles * 8 < p.rows * parts) col_tiles *= 2;
    for (;; col_tiles /= 2) {
        if (col_tiles == 0) return false;
        q.row_tile = col_tiles * 8 / parts;
        if (q.row_tile > p.rows) q.row_tile = p.rows;
        q.tiles = (p.out_features - 1) / (16 * mats(col_tiles)) + 1;
        // The split whose waves of tiles take the least, in steps of a warp: a tile ends
        // with about one step's time for its parts' addition, two in a cluster.
        Plan best = {};
        double least = 0.0;
        for (q.split = 1; q.split <= 8 && q.split <= q.steps; q.split *= 2) {
            const int slice = (q.steps - 1) / q.split + 1;
            q.warps = slice < kMaxWarps ? slice : kMaxWarps;
            lay_out(q, col_tiles, blocks);
            if (q.smem > kSmemLimit) continue;
            const int fit = kSmemLimit / (q.smem + 1024), most = ctas(col_tiles) * kMaxWarps / q.warps;
            const int resident = fit < 1 ? 1 : fit < most ? fit : most;
            q.clusters = 152 * resident / q.split;
            if (q.clusters > q.tiles) q.clusters = q.tiles;
            const int each = (q.tiles - 1) / q.clusters + 1;
            q.clusters = (q.tiles - 1) / each + 1;
            const int busy = (q.clusters * q.split - 1) / 152 + 1;      // CTAs of an SM
            const int side = busy * q.warps < 16 ? 16 : busy * q.warps;     // fewer warps do not take their steps faster
            const double cost = side * each * (q.per_warp + (q.split > 1 ? 2.0 : 1.0)) + busy * slice * q.row_tile * parts * 0.25;
            if (best.split == 0 || cost < least) {
                best = q;
                least = cost;
            }
        }
        if (best.split != 0) {
            q = best;
            break;
        }
    }
    if ((p.rows - 1) / q.row_tile + 1 > 65535) return false;
    *error = col_tiles == 1   ? run<1>(q, blocks, stream)
             : col_tiles == 2 ? run<2>(q, blocks, stream)
             : col_tiles == 4 ? run<4>(q, blocks, stream)
                              : run<8>(q, blocks, stream);
    return true;
}

}  // namespace ssd
