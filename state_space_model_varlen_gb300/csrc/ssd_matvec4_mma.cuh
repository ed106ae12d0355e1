// Products of few rows with 4-bit weights on the tensor cores.  One translation unit
// for each number of columns of a pass.
//
// A warp multiplies 32 (16 for many columns) outputs by 128 columns of x at a step
// (mma.m16n8k16, weights as its 16 rows, rows of x as its columns).  (code - zero) / 64
// is exact in bf16, as are 8-bit activations; fp32 activations become three bf16 parts
// of eight bits each, which together are exact.  Sums within a group are the
// instruction's fp32 sums; the groups' scales, times 64, are applied to them in fp32.
//
// Bound by HBM in principle, by latency in fact, at the 9 to 16 warps an SM that two
// CTAs make; no pipe is full.  One row of 4,096 to 18,560 issues in 47 % of the cycles (the
// integer pipe is 38 % busy) and waits at the chunk's barrier, for fixed latencies and for
// the first codes; 16 rows with groups of 32 in 36 % (25), 166 CTAs where 304 have room; the
// head of 2^17 outputs in 61 % (50) while its 512 CTAs, 1.7 rounds of those places, run.
// A step of 32 outputs x 128 columns is about 300 instructions, of which 160 unpack the
// codes and 16 are products (these alone ran at 8.1 TB/s of codes with 8 warps an SM).  Codes stream through a ring of asynchronous copies
// of each warp's own, a few steps deep.  x and the scales come through two buffers in
// shared memory, a chunk of steps ahead in registers.  Where there are few tiles two or
// four warps take the steps of the same outputs in turn, and a cluster of CTAs shares a
// tile's columns; the parts are added in a fixed order.
//
// Measured (floor at the copy rate): 1 row of 4,096 to 18,560 outputs, groups of 128,
// 12.0 us (5.8); 3 rows of 4,096 to 131,072 61.7 us (41); 16 rows of 2,560 to 10,576,
// groups of 32 with zeros, 16.4 us (2.4; scales and zeros of every block besides).  Rows of 4,102 columns, which no 16-byte copy takes whole, 29 us where rows
// of 4,096 take 12; 16 rows 17 us, 32 26, 64 44.  Before: tiles of 32 outputs whose columns
// eight warps shared, all of x in shared memory (head 63 us; 22 to 29 us where x of many
// rows left one CTA an SM, and whole rows alone); codes shifted to the mantissa's end and
// 128 + zero subtracted (three shifts a word for one: 73 for 69 us); 64 columns a pass
// with one CTA an SM (64 rows 56 for 51 us); the parts added one output at a time (16 rows
// 19.7 for 16.9).
//
// A group of columns is taken in blocks of 32; a group of another size, or a row's
// end, leaves the last block's x partly zero.  Rows of codes in whole 16 bytes are
// copied as they are (kWhole); of others the two 16-byte pieces that hold a block are,
// and its bytes are picked out of them.
#pragma once

#include <type_traits>

#include "ssd_layer_internal.h"
#include "ssd_mixer_common.cuh"

namespace ssd {

struct Matvec4Plan {
    ssd_matvec4_params p;
    int row_tile;               // rows of x of a pass
    int split;                  // CTAs of a cluster
    int ways;                   // warps that share outputs: 1, 2 or 4, at most the steps of a chunk
    int tiles;                  // of outputs
    int blocks, steps;          // of a row: 32 columns at most, four blocks
    int groups, x_groups;       // of a row
    int group_blocks, x_group_blocks;           // blocks of a group
    uint32_t group_magic, x_group_magic;        // floor(2^32 / blocks of a group) + 1
    int padded;                 // columns of a group that are not whole blocks, or 0
    int x_rows;                 // rows of x (their parts) in shared memory
    int off_x, off_scale, off_zero, off_xs, smem;
};

// for passes of 8, 16 and 32 columns; shared: blocks that share their scales (1, 2, 4)
cudaError_t launch_matvec4_cols1(const Matvec4Plan &q, int shared, bool whole, cudaStream_t stream);
cudaError_t launch_matvec4_cols2(const Matvec4Plan &q, int shared, bool whole, cudaStream_t stream);
cudaError_t launch_matvec4_cols4(const Matvec4Plan &q, int shared, bool whole, cudaStream_t stream);

namespace matvec4 {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kStep = 128, kSmemLimit = 227 * 1024;
constexpr int mats(int cols) { return cols <= 2 ? 2 : 1; }          // sixteens of outputs of a warp
constexpr int chunk(int cols, int shared) { return cols == 1 && shared == 4 ? 4 : 2; }    // steps of a buffer of x and scales
// steps of codes in the ring of a warp: what two CTAs an SM leave room for
constexpr int stages(int shared, bool whole) { return !whole ? 2 : shared == 4 ? 4 : 3; }
constexpr int kCtas = 2;                                            // of an SM, for the registers
constexpr int outs(int cols) { return kWarps * 16 * mats(cols); }   // of a tile
constexpr int scale_line(int cols) { return outs(cols) + 4; }       // a gap: the scales of an output come from lanes side by side
// bytes of a row of a stage: whole steps, with a gap where lanes read one another's; or two pieces a block
constexpr int pitch(int shared, bool whole) { return whole ? (shared == 4 ? 64 : 80) : 144; }
constexpr int x_pitch(int cols, int shared) { return chunk(cols, shared) * kStep * 2 + 64; }    // two rows beside one another in the banks

__host__ __device__ __forceinline__ int group_of(int block, int blocks, uint32_t magic) {
    return blocks == 1 ? block : (int)(((uint64_t)(uint32_t)block * magic) >> 32);
}

#ifdef __CUDACC__
namespace {

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

// v in a register, which the compiler does not load or compute again at each use
__device__ __forceinline__ int kept(int v) {
    int r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Codes i and i + 4 of a word (at bits 4 i and 4 i + 16) less their zero, over 64, as
// bf16: the low eight bits of a bf16 number without exponent bits above them are its
// value in units of 2^-133, subnormal or not, so that codes at bits 0 and 4 need no
// shift.  powers[i & 1] is 2^127 or 2^123, twice; zero is -zero / 64, twice.  Exact.
__device__ __forceinline__ uint32_t codes2(uint32_t word, int i, const uint32_t (&powers)[2], uint32_t zero) {
    const uint32_t v = (i >= 2 ? word >> 8 : word) & (i & 1 ? 0x00f000f0u : 0x000f000fu);
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(powers[i & 1]), "r"(zero));
    return r;
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Eight consecutive values of kSize bytes of a row of x as they are stored, by loads of
// at most 4 bytes, of which `grain` is the alignment; zeros behind the first `live`.
struct Raw { uint32_t w[8]; };
template <int kSize> __device__ __forceinline__ Raw load8(const uint8_t *src, int live, int grain) {
    Raw r{};
    if (live == 8 && grain >= 4) {
#pragma unroll
        for (int i = 0; i < 2 * kSize; ++i) r.w[i] = reinterpret_cast<const uint32_t *>(src)[i];
    } else if (kSize == 1 && live == 8 && grain == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(src)[i] << (16 * (i & 1));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= live) continue;
            if constexpr (kSize == 4) r.w[i] = reinterpret_cast<const uint32_t *>(src)[i];
            else if constexpr (kSize == 2) r.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(src)[i] << (16 * (i & 1));
            else r.w[i / 4] |= (uint32_t)src[i] << (8 * (i & 3));
        }
    }
    return r;
}
// the upper halves of a and b
__device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
// bf16 values of 8-bit codes, i and i + 4 side by side
template <int kType> __device__ __forceinline__ uint4 side_by_side(const uint4 &r) {
    float v[8];
    decode4<kType>(r.x, v);
    decode4<kType>(r.y, v + 4);
    return make_uint4(upper(__float_as_uint(v[0]), __float_as_uint(v[4])), upper(__float_as_uint(v[1]), __float_as_uint(v[5])),
                      upper(__float_as_uint(v[2]), __float_as_uint(v[6])), upper(__float_as_uint(v[3]), __float_as_uint(v[7])));
}

// kCols: eights of columns (rows of x, or their parts) of a pass.  kShared: blocks that
// certainly share their scales (1, 2, or 4: a step).
template <int kCols, int kShared, bool kZero, bool kWhole>
__global__ void __launch_bounds__(kThreads, kCtas) matvec4_mma_kernel(const __grid_constant__ Matvec4Plan plan) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kMats = mats(kCols), kRows = 16 * kMats, kOuts = outs(kCols), kChunk = chunk(kCols, kShared);
    constexpr int kStages = stages(kShared, kWhole);
    constexpr int kPitch = pitch(kShared, kWhole), kStageBytes = kRows * kPitch, kXPitch = x_pitch(kCols, kShared);
    constexpr int kFlushes = 4 / kShared, kScales = kChunk * kFlushes;  // of a step, of a chunk
    constexpr int kScaleLine = scale_line(kCols);
    // eights of x that a thread brings of a chunk, and of them in fp32, which take two registers' places
    constexpr int kEights = kChunk * 16, kNext = kThreads / kEights;
    constexpr int kItems = kCols * 8 / kNext, kItems32 = (kCols * 8 / 3 - 1) / kNext + 1;
    constexpr int kRaw = kItems > 2 * kItems32 ? kItems : 2 * kItems32;
    constexpr bool kOwn = kWhole && kShared == 4;                       // a lane reads the codes that it copied itself
    const ssd_matvec4_params &p = plan.p;
    const int thread = kept(threadIdx.x), lane = thread & 31, g = lane >> 2, t = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, thread >> 5, 0);          // known to be the same in all lanes
    const uint32_t powers[2] = {(uint32_t)kept(0x7f007f00), (uint32_t)kept(0x7d007d00)};
    const uint32_t eight = (uint32_t)kept((int)0xbe00be00u);            // -8 / 64, twice
    const int ways = kChunk > 1 ? plan.ways : 1, turn = warp & (ways - 1);
    const int outs_now = kOuts / ways;                                  // of the tile
    const int rank = blockIdx.x % plan.split, tile = blockIdx.x / plan.split;
    const int r0 = blockIdx.y * plan.row_tile, rows = min(plan.row_tile, p.rows - r0);
    const int parts = p.x_dtype == SSD_F32 ? 3 : 1, cols = rows * parts;
    const int chunks = (plan.steps - 1) / kChunk + 1;
    const int chunk0 = (int)((int64_t)chunks * rank / plan.split), chunk1 = (int)((int64_t)chunks * (rank + 1) / plan.split);
    const int step0 = chunk0 * kChunk, step1 = min(plan.steps, chunk1 * kChunk);
    const int o_first = (kChunk > 1 ? warp / ways : warp) * kRows;     // of the warp's in the tile
    const int64_t o_tile = (int64_t)tile * outs_now, o_warp = o_tile + o_first;
    const bool busy = o_warp < p.out_features;                          // the warp has outputs
    const bool x8 = p.x_scale != nullptr && plan.x_groups > 1;          // one scale of a whole row is applied at the end
    uint8_t *const ring = smem + warp * (kStages * kStageBytes);
    await_previous();

    // first column of a block, and the end of the columns that are its
    auto columns = [&](int block, int &end) {
        if (plan.padded == 0) {
            end = p.in_features;
            return block * 32;
        }
        const int group = group_of(block, plan.group_blocks, plan.group_magic);
        end = min(p.in_features, (group + 1) * plan.padded);
        return group * plan.padded + (block - group * plan.group_blocks) * 32;
    };

    // ---- codes ----
    const uint8_t *src[2 * kMats];                      // rows g + 8 h: of the lane's 16 bytes (kWhole), or their beginning
#pragma unroll
    for (int h = 0; h < 2 * kMats; ++h)
        src[h] = p.weight + min(o_warp + g + 8 * h, (int64_t)p.out_features - 1) * p.weight_stride;
    const uint8_t *const last_row = p.weight + (int64_t)(p.out_features - 1) * p.weight_stride;
    const uint8_t *const codes_end = last_row + (p.in_features + 1) / 2;
    const uint8_t *const piece_src = p.weight + (o_warp + (lane >> 3)) * p.weight_stride;
    int to_step = step0 + turn, to_stage = 0;
    const int row_bytes = kept(p.in_features / 2), whole_steps = kept(p.in_features / kStep);
    auto issue = [&]() {
        if (busy && to_step < step1) {
            uint8_t *const dst = ring + to_stage * kStageBytes;
            if constexpr (kWhole) {
                const int byte = to_step * (kStep / 2) + t * 16;
                const bool live = to_step < whole_steps || byte < row_bytes;
#pragma unroll
                for (int h = 0; h < 2 * kMats; ++h)
                    copy_async<16>(dst + (g + 8 * h) * kPitch + t * 16, src[h] + (live ? byte : 0), live);
            } else {
                // 4 rows x 4 blocks x 2 pieces at a time; pieces that pass the matrix's ends byte by byte
                const int block = to_step * 4 + (lane >> 1 & 3);
                uint8_t *to = dst + (lane >> 3) * kPitch + (lane & 7) * 16;
                if (block >= plan.blocks) {
#pragma unroll
                    for (int i = 0; i < kRows / 4; ++i, to += 4 * kPitch) *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
                } else {
                    int stop;
                    const int off = columns(block, stop) / 2;
                    const uint8_t *row = piece_src + off;
                    int64_t o = o_warp + (lane >> 3);
#pragma unroll 4
                    for (int i = 0; i < kRows / 4; ++i, to += 4 * kPitch, o += 4, row += 4 * p.weight_stride) {
                        const uint8_t *from = o < p.out_features ? row : last_row + off;
                        from += (lane & 1) * 16 - (int)(reinterpret_cast<uintptr_t>(from) & 15);
                        if (from >= p.weight && from + 16 <= codes_end) {
                            copy_async<16>(to, from, true);
                        } else {
                            for (int b = 0; b < 16; ++b) to[b] = from + b >= p.weight && from + b < codes_end ? from[b] : 0;
                        }
                    }
                }
            }
        }
        to_step += ways;
        to_stage = to_stage + 1 == kStages ? 0 : to_stage + 1;
        commit_async();
    };
    // ---- x and scales: a chunk's into registers, and from there into a buffer ----
    const int x_elem = p.x_dtype == SSD_F32 ? 4 : p.x_dtype == SSD_BF16 ? 2 : 1;
    const int x_low = (int)(reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)(p.x_stride * x_elem) | (uintptr_t)(plan.padded * x_elem));
    const int x_grain = x_low % (x_elem == 1 ? 8 : 16) == 0 ? 16 : x_low % 4 == 0 ? 4 : x_low % 2 == 0 ? 2 : 1;
    const int scale_f = thread % kScales, scale_row = thread / kScales;         // the first scale that the thread brings
    const int scale_rows = (int)min((int64_t)outs_now, p.out_features - o_tile);
    // eights of x that the thread brings: one place in the chunk, of every kNext-th row
    const int x_e = thread % kEights, x_row = thread / kEights;
    const uint8_t *const x_src = static_cast<const uint8_t *>(p.x) + (int64_t)(r0 + x_row) * p.x_stride * x_elem;
    const int64_t x_next = (int64_t)kNext * p.x_stride * x_elem;
    const uint8_t *const scale_src =
        static_cast<const uint8_t *>(p.scale) + (o_tile + scale_row) * plan.groups * (p.scale_dtype == SSD_F32 ? 4 : 2);
    const uint8_t *const zero_src = kZero ? p.zero + (o_tile + scale_row) * plan.groups : nullptr;
    const int scale_next = kThreads / kScales;
    uint4 x_raw[kRaw];          // item i at i, or in fp32 at 2 i and 2 i + 1
    uint32_t scale_raw[kScales], zero_raw[kScales];
    constexpr int kXScales = (kScales * kCols * 8 - 1) / kThreads + 1;
    float xs_raw[kXScales];
    auto bring = [&](int c) {
        {
            const int block = c * kChunk * 4 + x_e / 4;
            int live = 0, k = 0;
            if (block < plan.blocks) {
                int end;
                k = columns(block, end) + (x_e & 3) * 8;
                live = max(0, min(8, end - k));
            }
            const uint8_t *from = x_src + (int64_t)k * x_elem;
            const bool wide = live == 8 && x_grain == 16;
            if (x_elem == 4) {
#pragma unroll
                for (int i = 0; i < kItems32; ++i, from += x_next) {
                    x_raw[2 * i] = x_raw[2 * i + 1] = make_uint4(0, 0, 0, 0);
                    if (x_row + i * kNext >= rows || live == 0) continue;
                    if (wide) {
                        x_raw[2 * i] = *reinterpret_cast<const uint4 *>(from);
                        x_raw[2 * i + 1] = *reinterpret_cast<const uint4 *>(from + 16);
                    } else {
                        const Raw r = load8<4>(from, live, x_grain);
                        x_raw[2 * i] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
                        x_raw[2 * i + 1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kItems; ++i, from += x_next) {
                    x_raw[i] = make_uint4(0, 0, 0, 0);
                    if (x_row + i * kNext >= rows || live == 0) continue;
                    if (!wide) {
                        const Raw r = x_elem == 2 ? load8<2>(from, live, x_grain) : load8<1>(from, live, x_grain);
                        x_raw[i] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
                    } else if (x_elem == 2) {
                        x_raw[i] = *reinterpret_cast<const uint4 *>(from);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(from);
                        x_raw[i].x = v.x;
                        x_raw[i].y = v.y;
                    }
                }
            }
        }
        {
            // neighbours take the scales of one output
            const int block = min(c * kChunk * 4 + scale_f * kShared, plan.blocks - 1);
            const int group = group_of(block, plan.group_blocks, plan.group_magic);
            if (p.scale_dtype == SSD_F32) {
                const uint8_t *from = scale_src + group * 4;
#pragma unroll
                for (int i = 0; i < kScales; ++i, from += (int64_t)scale_next * plan.groups * 4)
                    if (scale_row + i * scale_next < scale_rows) scale_raw[i] = *reinterpret_cast<const uint32_t *>(from);
            } else {
                const uint8_t *from = scale_src + group * 2;
#pragma unroll
                for (int i = 0; i < kScales; ++i, from += (int64_t)scale_next * plan.groups * 2)
                    if (scale_row + i * scale_next < scale_rows) scale_raw[i] = *reinterpret_cast<const uint16_t *>(from);
            }
            if constexpr (kZero) {
                const uint8_t *from = zero_src + group;
#pragma unroll
                for (int i = 0; i < kScales; ++i, from += (int64_t)scale_next * plan.groups)
                    if (scale_row + i * scale_next < scale_rows) zero_raw[i] = *from;
            }
        }
        if (x8)
#pragma unroll
            for (int i = 0; i < kXScales; ++i) {
                const int item = thread + i * kThreads, col = item % (kCols * 8), f = item / (kCols * 8);
                xs_raw[i] = 0.f;
                if (f >= kScales || col >= rows) continue;
                const int group = group_of(min(c * kChunk * 4 + f * kShared, plan.blocks - 1), plan.x_group_blocks, plan.x_group_magic);
                xs_raw[i] = p.x_scale[(int64_t)(r0 + col) * plan.x_groups + group];
            }
    };
    auto put_away = [&](int buffer) {
        // values i and i + 4 side by side, as the codes of a word come; eights of a step
        // in the order in which quad lane t reads its j-th word: 4 j + t
        const int place = kOwn ? (x_e & ~15) | (x_e & 3) << 2 | (x_e >> 2 & 3) : x_e;
        uint8_t *const xs = smem + plan.off_x + buffer * (plan.x_rows * kXPitch) + x_row * kXPitch + place * 16;
        auto each = [&](auto eight) {
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (x_row + i * kNext < rows) *reinterpret_cast<uint4 *>(xs + i * kNext * kXPitch) = eight(x_raw[i]);
        };
        if (p.x_dtype == SSD_BF16) {
            each([](const uint4 &r) {
                return make_uint4(__byte_perm(r.x, r.z, 0x5410), upper(r.x, r.z), __byte_perm(r.y, r.w, 0x5410), upper(r.y, r.w));
            });
        } else if (p.x_dtype == SSD_E4M3) {
            each([](const uint4 &r) { return side_by_side<SSD_E4M3>(r); });
        } else if (p.x_dtype == SSD_I8) {
            each([](const uint4 &r) { return side_by_side<SSD_I8>(r); });
        } else {
#pragma unroll
            for (int i = 0; i < kItems32; ++i) {
                if (x_row + i * kNext >= rows) continue;
                const uint4 lo = x_raw[2 * i], hi = x_raw[2 * i + 1];
                float v[8] = {__uint_as_float(lo.x), __uint_as_float(lo.y), __uint_as_float(lo.z), __uint_as_float(lo.w),
                              __uint_as_float(hi.x), __uint_as_float(hi.y), __uint_as_float(hi.z), __uint_as_float(hi.w)};
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    uint32_t u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {       // the upper bits, and what is left of a finite number
                        u[j] = v[j] != v[j] ? 0x7fc00000u : __float_as_uint(v[j]);
                        const float cut = __uint_as_float(u[j] & 0xffff0000u);
                        v[j] = fabsf(cut) < __int_as_float(0x7f800000) ? v[j] - cut : 0.f;
                    }
                    *reinterpret_cast<uint4 *>(xs + (i * kNext + part * rows) * kXPitch) =
                        make_uint4(upper(u[0], u[4]), upper(u[1], u[5]), upper(u[2], u[6]), upper(u[3], u[7]));
                }
            }
        }
        float *const scales = reinterpret_cast<float *>(smem + plan.off_scale) + (buffer * kScales + scale_f) * kScaleLine + scale_row;
        uint32_t *const zeros = reinterpret_cast<uint32_t *>(smem + plan.off_zero) + (buffer * kScales + scale_f) * kScaleLine + scale_row;
        auto put_scales = [&](auto value) {
#pragma unroll
            for (int i = 0; i < kScales; ++i)
                if (scale_row + i * scale_next < scale_rows) scales[i * scale_next] = 64.f * value(scale_raw[i]);
        };
        if (p.scale_dtype == SSD_F32) put_scales([](uint32_t v) { return __uint_as_float(v); });
        else if (p.scale_dtype == SSD_BF16) put_scales([](uint32_t v) { return __uint_as_float(v << 16); });
        else put_scales([](uint32_t v) { return __half2float(__ushort_as_half((unsigned short)v)); });
        if constexpr (kZero) {
#pragma unroll
            for (int i = 0; i < kScales; ++i)
                if (scale_row + i * scale_next < scale_rows)
                    zeros[i * scale_next] = (__float_as_uint((float)zero_raw[i] * -0.015625f) >> 16) * 0x00010001u;
        }
        if (x8)
#pragma unroll
            for (int i = 0; i < kXScales; ++i)
                if (thread + i * kThreads < kScales * kCols * 8)
                    reinterpret_cast<float *>(smem + plan.off_xs)[buffer * (kScales * kCols * 8) + thread + i * kThreads] = xs_raw[i];
    };

    bring(chunk0);
#pragma unroll 1
    for (int q = 0; q < kStages - 1; ++q) issue();
    put_away(0);
    __syncthreads();

    // A column that is not there is computed from the last one and not looked at.
    int x_at[kCols];
#pragma unroll
    for (int n = 0; n < kCols; ++n) x_at[n] = plan.off_x + min(n * 8 + g, cols - 1) * kXPitch + t * 16;
    float sum[kMats][kCols][4];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[m][n][i] = 0.f;
    int stage = 0, buffer = 0;
#pragma unroll 1
    for (int c = chunk0; c < chunk1; ++c) {
        if (c + 1 < chunk1) bring(c + 1);
        const uint8_t *const x_now = smem + buffer * (plan.x_rows * kXPitch);
        const float *const scales = reinterpret_cast<const float *>(smem + plan.off_scale) + buffer * (kScales * kScaleLine) + o_first + g;
        const uint32_t *const zeros = reinterpret_cast<const uint32_t *>(smem + plan.off_zero) + buffer * (kScales * kScaleLine) + o_first + g;
        const float *const x_scales = reinterpret_cast<const float *>(smem + plan.off_xs) + buffer * (kScales * kCols * 8) + 2 * t;
#pragma unroll 1
        for (int s = turn; s < kChunk; s += ways) {
            const int step = c * kChunk + s;
            if (!busy || step >= step1) break;
            wait_async<kStages - 2>();
            if constexpr (!kOwn) __syncwarp();          // a lane reads what its neighbours copied
            issue();
            const uint8_t *const codes = ring + stage * kStageBytes + g * kPitch + (kOwn ? t * 16 : t * 4);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            const float *const s_scales = scales + s * (kFlushes * kScaleLine), *const s_x = x_scales + s * (kFlushes * kCols * 8);
            const uint32_t *const s_zeros = zeros + s * (kFlushes * kScaleLine);
            const uint8_t *x[kCols];
#pragma unroll
            for (int n = 0; n < kCols; ++n) x[n] = x_now + s * (kStep * 2) + x_at[n];
            const int flushes = kFlushes == 1 ? 1 : min(kFlushes, (plan.blocks - step * 4 + kShared - 1) / kShared);
            uint32_t words[2 * kMats][4];
            if constexpr (kOwn) {
#pragma unroll
                for (int h = 0; h < 2 * kMats; ++h)
                    *reinterpret_cast<uint4 *>(words[h]) = *reinterpret_cast<const uint4 *>(codes + 8 * h * kPitch);
            }
#pragma unroll
            for (int f = 0; f < kFlushes; ++f) {
                if (f >= flushes) break;
                uint32_t zero[2 * kMats];               // -zero / 64, twice
#pragma unroll
                for (int h = 0; h < 2 * kMats; ++h) zero[h] = kZero ? s_zeros[f * kScaleLine + 8 * h] : eight;
                float acc[kMats][kCols][4];
#pragma unroll
                for (int b = 0; b < kShared; ++b) {
                    const int w = f * kShared + b;
                    uint32_t a0[kMats][4], a1[kMats][4];
                    int shift = 0;
                    if constexpr (!kWhole) {
                        int stop;
                        shift = columns(min(step * 4 + w, plan.blocks - 1), stop) / 2;
                    }
#pragma unroll
                    for (int m = 0; m < kMats; ++m) {
                        uint32_t pair[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (kOwn) {
                                pair[h] = words[2 * m + h][w];
                            } else if constexpr (kWhole) {
                                pair[h] = *reinterpret_cast<const uint32_t *>(codes + (16 * m + 8 * h) * kPitch + w * 16);
                            } else {
                                const int off = (int)((reinterpret_cast<uintptr_t>(src[2 * m + h]) + shift) & 15);
                                const uint8_t *at = codes + (16 * m + 8 * h) * kPitch + w * 32 + (off & ~3);
                                pair[h] = __funnelshift_r(*reinterpret_cast<const uint32_t *>(at), *reinterpret_cast<const uint32_t *>(at + 4),
                                                          8 * (off & 3));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            a0[m][2 * i] = codes2(pair[0], i, powers, zero[2 * m]);
                            a0[m][2 * i + 1] = codes2(pair[1], i, powers, zero[2 * m + 1]);
                            a1[m][2 * i] = codes2(pair[0], i + 2, powers, zero[2 * m]);
                            a1[m][2 * i + 1] = codes2(pair[1], i + 2, powers, zero[2 * m + 1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kCols; ++n) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(x[n] + w * 64);
#pragma unroll
                        for (int m = 0; m < kMats; ++m) {
                            if (b == 0) mma_first(acc[m][n], a0[m], v.x, v.y);
                            else mma(acc[m][n], a0[m], v.x, v.y);
                            mma(acc[m][n], a1[m], v.z, v.w);
                        }
                    }
                }
                float scale[2 * kMats];
#pragma unroll
                for (int h = 0; h < 2 * kMats; ++h) scale[h] = s_scales[f * kScaleLine + 8 * h];
#pragma unroll
                for (int n = 0; n < kCols; ++n) {
                    if (x8) {
                        const float2 u = *reinterpret_cast<const float2 *>(s_x + f * (kCols * 8) + n * 8);
#pragma unroll
                        for (int m = 0; m < kMats; ++m) {
                            acc[m][n][0] *= u.x;
                            acc[m][n][1] *= u.y;
                            acc[m][n][2] *= u.x;
                            acc[m][n][3] *= u.y;
                        }
                    }
#pragma unroll
                    for (int m = 0; m < kMats; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[m][n][i] = fmaf(acc[m][n][i], scale[2 * m + i / 2], sum[m][n][i]);
                }
            }
        }
        buffer ^= 1;
        if (c + 1 < chunk1) put_away(buffer);
        __syncthreads();
    }

    // The sums, through shared memory (everything there has been read): [column][output].
    const int line = outs_now + 4;
    float *const own = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = n * 8 + 2 * t + (i & 1);
                if (col < cols) own[(turn * cols + col) * line + o_first + 16 * m + g + 8 * (i >> 1)] = sum[m][n][i];
            }
    if (plan.split > 1) cluster_barrier();
    else __syncthreads();
    // four outputs of a row at a time
    const uint32_t local = (uint32_t)__cvta_generic_to_shared(own);
    const int fours = outs_now / 4, log_fours = __ffs(fours) - 1;
    const bool out_wide = p.out_stride % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % (p.out_dtype == SSD_F32 ? 16 : 8) == 0;
    for (int i = rank * kThreads + thread; i < rows * fours; i += plan.split * kThreads) {
        const int r = i >> log_fours, o = (i & (fours - 1)) * 4;
        const int live = (int)min((int64_t)4, p.out_features - o_tile - o);
        if (live <= 0) continue;
        float v[4] = {};
        for (int c = 0; c < plan.split; ++c) {
            uint32_t at = local + (r * line + o) * 4;
            if (plan.split > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(at), "r"(c));
            for (int part = 0; part < parts * ways; ++part) {
                float4 f;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(at + part * rows * (line * 4)) : "memory");
                v[0] += f.x;
                v[1] += f.y;
                v[2] += f.z;
                v[3] += f.w;
            }
        }
        if (p.x_scale != nullptr && plan.x_groups == 1) {
            const float scale = p.x_scale[r0 + r];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] *= scale;
        }
        const int64_t at = (int64_t)(r0 + r) * p.out_stride + o_tile + o;
        auto finish = [&](auto *out, const auto *bias) {
            using T = std::remove_reference_t<decltype(*out)>;
            Pack<T, 4> q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (bias && j < live) v[j] += to_float(bias[o_tile + o + j]);
                q.v[j] = from_float<T>(v[j]);
            }
            if (live == 4 && out_wide) {
                store_pack<T, 4>(out + at, q);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < live) out[at + j] = q.v[j];
            }
        };
        if (p.out_dtype == SSD_F32) finish(static_cast<float *>(p.out), static_cast<const float *>(p.bias));
        else finish(static_cast<__nv_bfloat16 *>(p.out), static_cast<const __nv_bfloat16 *>(p.bias));
    }
    if (plan.split > 1) cluster_barrier();              // no CTA leaves while another reads its sums
}

template <int kCols, int kShared, bool kZero, bool kWhole> cudaError_t run(const Matvec4Plan &q, cudaStream_t stream) {
    auto f = matvec4_mma_kernel<kCols, kShared, kZero, kWhole>;
    // the most that any plan takes, so that one call of a process and device is enough
    static unsigned long long set = 0;          // bit d: device d (the first 64)
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= 64 || !(__atomic_load_n(&set, __ATOMIC_ACQUIRE) >> device & 1)) {
        e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
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
    config.gridDim = dim3((unsigned)(q.tiles * q.split), (unsigned)((q.p.rows - 1) / q.row_tile + 1));
    config.blockDim = dim3(kThreads);
    config.dynamicSmemBytes = (size_t)q.smem;
    config.stream = stream;
    config.attrs = attr;
    config.numAttrs = q.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&config, f, q);
}

template <int kCols, int kShared> cudaError_t run(const Matvec4Plan &q, bool whole, cudaStream_t stream) {
    if (q.p.zero) return whole ? run<kCols, kShared, true, true>(q, stream) : run<kCols, kShared, true, false>(q, stream);
    return whole ? run<kCols, kShared, false, true>(q, stream) : run<kCols, kShared, false, false>(q, stream);
}

template <int kCols> cudaError_t run(const Matvec4Plan &q, int shared, bool whole, cudaStream_t stream) {
    return shared == 4   ? run<kCols, 4>(q, whole, stream)
           : shared == 2 ? run<kCols, 2>(q, whole, stream)
                         : run<kCols, 1>(q, whole, stream);
}

}  // namespace
#endif
}  // namespace matvec4
}  // namespace ssd
