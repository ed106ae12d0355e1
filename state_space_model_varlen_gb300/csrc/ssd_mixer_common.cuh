// Device helpers of the mixer operators: element and vector access, the
// activations, and the storage of state rows (8-bit codes among them).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ssd_mixer.h"
#include "ssd_common.cuh"

namespace ssd {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// First statement of every kernel: waits until all work before it in the stream
// is done and visible.  (No kernel lets the next one start early: its CTAs then
// held places of this one's, 20.6 for 19.7 us of two convolutions back to back.)
__device__ __forceinline__ void await_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// V consecutive elements moved together (one instruction up to 16 bytes).
constexpr int pack_align(int bytes) { return bytes % 16 == 0 ? 16 : bytes & -bytes; }
template <typename T, int V> struct alignas(pack_align(sizeof(T) * V)) Pack { T v[V]; };

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T *src) {
    return *reinterpret_cast<const Pack<T, V> *>(src);
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T *dst, const Pack<T, V> &p) {
    *reinterpret_cast<Pack<T, V> *>(dst) = p;
}

// kBytes (4, 8 or 16) from global to shared memory, asynchronously; zeros where
// `live` is false (src is then any valid address, not read).  A thread that
// reads its own copies back needs no barrier, only wait_async.
template <int kBytes>
__device__ __forceinline__ void copy_async(void *dst, const void *src, bool live) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    const int n = live ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(src), "n"(kBytes), "r"(n) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the thread's newest kPending groups of copies have landed
template <int kPending> __device__ __forceinline__ void wait_async() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// v sigmoid(v) through the ex2 and rcp approximations, four instructions where
// expf and a division take many: relative error below 2^-20 + |v| 2^-23, the
// second part from the rounding of the exponent v log2(e) (2^-18 at v = -30).
// Below about v = -87.3, where the result is below 2^-119, the reciprocal is
// flushed and the result is zero.
__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float silu(float v) { return v * rcp_approx(1.f + ex2_approx(v * -1.4426950408889634f)); }

// v / (1 + e^-v), each operation rounded by itself
__device__ __forceinline__ float silu_stepwise(float v) { return __fdiv_rn(v, __fadd_rn(1.f, expf(-v))); }

// softplus(z) = log(1 + e^z) in the overflow-safe form max(z,0) + log1p(e^-|z|)
__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// Two fp32 operations in one instruction.  (ptxas merges a packed product and a
// packed sum into one fused operation; where the product's own rounding
// matters, the sum is two scalar __fadd_rn.)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r, x, y, z;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    memcpy(&z, &c, 8);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    float2 o;
    memcpy(&o, &r, 8);
    return o;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r, x, y;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 o;
    memcpy(&o, &r, 8);
    return o;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r, x, y;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 o;
    memcpy(&o, &r, 8);
    return o;
}
__device__ __forceinline__ float2 silu2(float2 v) {
    const float2 e = mul2(v, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 d = add2(make_float2(ex2_approx(e.x), ex2_approx(e.y)), make_float2(1.f, 1.f));
    return mul2(v, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
}

// Elements 2 i, 2 i + 1 of a pack as floats, and back.
template <int V> __device__ __forceinline__ float2 pair_of(const Pack<float, V> &p, int i) {
    return make_float2(p.v[2 * i], p.v[2 * i + 1]);
}
template <int V> __device__ __forceinline__ float2 pair_of(const Pack<__nv_bfloat16, V> &p, int i) {
    uint32_t w;
    memcpy(&w, p.v + 2 * i, 4);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int V> __device__ __forceinline__ void set_pair(Pack<float, V> &p, int i, float2 f) {
    p.v[2 * i] = f.x;
    p.v[2 * i + 1] = f.y;
}
template <int V> __device__ __forceinline__ void set_pair(Pack<__nv_bfloat16, V> &p, int i, float2 f) {
    const __nv_bfloat162 b = __float22bfloat162_rn(f);
    memcpy(p.v + 2 * i, &b, 4);
}

// ---------------------------------------------------------------------------
// state storage
// ---------------------------------------------------------------------------
template <int kType> struct Stored;          // kType: SSD_F32, SSD_BF16, SSD_F16, SSD_E4M3, SSD_I8
template <> struct Stored<SSD_F32> { using T = float; };
template <> struct Stored<SSD_BF16> { using T = __nv_bfloat16; };
template <> struct Stored<SSD_F16> { using T = __half; };
template <> struct Stored<SSD_E4M3> { using T = uint8_t; };
template <> struct Stored<SSD_I8> { using T = uint8_t; };

// Largest code of the 8-bit types.
template <int kType> constexpr float code_limit() { return kType == SSD_I8 ? 127.f : 448.f; }

// Four codes, packed low to high, as floats without their scale.
template <int kType> __device__ __forceinline__ void decode4(uint32_t w, float *out) {
    if constexpr (kType == SSD_E4M3) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
        __half2 h0, h1;
        memcpy(&h0, &lo, 4);
        memcpy(&h1, &hi, 4);
        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
        out[0] = f0.x;
        out[1] = f0.y;
        out[2] = f1.x;
        out[3] = f1.y;
    } else {
        // the code + 128 as the low byte of 2^23's mantissa
        w ^= 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | i)) - 8388736.f;
    }
}

// Stored values as floats; 8-bit codes without their scale.
template <int kType, int V>
__device__ __forceinline__ void decode(const Pack<typename Stored<kType>::T, V> &p, float *out) {
    if constexpr ((kType == SSD_E4M3 || kType == SSD_I8) && V >= 4) {
        uint32_t w[V / 4];
        memcpy(w, p.v, V);
#pragma unroll
        for (int j = 0; j < V; j += 4) decode4<kType>(w[j / 4], out + j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (kType == SSD_F32) out[j] = p.v[j];
            else if constexpr (kType == SSD_BF16) out[j] = __bfloat162float(p.v[j]);
            else if constexpr (kType == SSD_F16) out[j] = __half2float(p.v[j]);
            else if constexpr (kType == SSD_E4M3)
                out[j] = __half2float(__half(__nv_cvt_fp8_to_halfraw(p.v[j], __NV_E4M3)));
            else
                out[j] = (float)(int8_t)p.v[j];
        }
    }
}

// What a row's largest magnitude makes of its scale: inv = (1 / m) limit, with
// both operations rounded, multiplies the values; scale multiplies the codes.
__device__ __forceinline__ void row_scale(float m, float limit, float *inv, float *scale) {
    *scale = __fmul_rn(m, 1.f / limit);
    if (!(m < __int_as_float(0x7f800000))) {            // an infinity or a NaN in the row
        *inv = 0.f;
        *scale = __int_as_float(0x7fffffff);
    } else if (m < 7.888609052210118e-31f) {            // 2^-100
        *inv = *scale = 0.f;
    } else {
        *inv = __fmul_rn(__frcp_rn(m), limit);
    }
}

// sr_f16 with the dropped part as an integer: where fp16 is normal,
// (|v| - |lo|) / spacing is the 13 dropped bits over 2^13; below, the fraction
// of |v| in units of 2^-24.  From 2^16 on (and for what is not finite) the general form.
static __device__ __noinline__ uint32_t sr_f16_large(float v, uint32_t r) { return __half_as_ushort(sr_f16(v, r)); }
__device__ __forceinline__ __half sr_f16_fast(float v, uint32_t r) {
    const uint32_t bits = __float_as_uint(v), a = bits & 0x7fffffffu, sign = bits >> 16 & 0x8000u;
    uint32_t h = ((a - 0x38000000u) >> 13) + ((a << 19) > r ? 1u : 0u) | sign;
    if (a < 0x38800000u) {                              // 2^-14
        const float u = __uint_as_float(a) * 16777216.f;
        const uint32_t lo = (uint32_t)u;
        h = lo + (__float2uint_ru((u - (float)lo) * 4294967296.f) > r ? 1u : 0u) | sign;
    } else if (a >= 0x47800000u) {
        h = sr_f16_large(v, r);
    }
    return __ushort_as_half((unsigned short)h);
}

// ---- nearest ---------------------------------------------------------------
template <int kType> __device__ __forceinline__ uint32_t encode4(const float *h, float inv) {
    if constexpr (kType == SSD_E4M3) {
        const float2 inv2 = make_float2(inv, inv);
        const float2 v0 = mul2(make_float2(h[0], h[1]), inv2), v1 = mul2(make_float2(h[2], h[3]), inv2);
        uint32_t w;
        asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}" : "=r"(w) : "f"(v0.x), "f"(v0.y), "f"(v1.x), "f"(v1.y));
        return w;
    } else {
        // 1.5 2^23 + v, whose rounding is the rounding to an integer
        const float2 inv2 = make_float2(inv, inv);
        const float2 lo = mul2(make_float2(h[0], h[1]), inv2), hi = mul2(make_float2(h[2], h[3]), inv2);
        const uint32_t t[4] = {__float_as_uint(__fadd_rn(lo.x, 12582912.f)), __float_as_uint(__fadd_rn(lo.y, 12582912.f)),
                               __float_as_uint(__fadd_rn(hi.x, 12582912.f)), __float_as_uint(__fadd_rn(hi.y, 12582912.f))};
        return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    }
}
template <int kType> __device__ __forceinline__ uint8_t encode1(float h, float inv) {
    const float v = __fmul_rn(h, inv);
    return kType == SSD_E4M3 ? (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3)
                             : (uint8_t)__float_as_uint(__fadd_rn(v, 12582912.f));
}

// V values times inv as codes, to nearest even.
template <int kType, int V>
__device__ __forceinline__ Pack<uint8_t, V> encode8(const float *h, float inv) {
    Pack<uint8_t, V> out;
    if constexpr (V >= 4) {
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V; j += 4) w[j / 4] = encode4<kType>(h + j, inv);
        memcpy(out.v, w, V);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out.v[j] = encode1<kType>(h[j], inv);
    }
    return out;
}

// ---- stochastic, see SSD_E4M3 in ssd_mixer.h ---------------------------------
// Random bytes of the 16 elements of block q: Philox as sr_block, with the ten
// rounds' keys prepared (keys[2 r], keys[2 r + 1]).
__device__ __forceinline__ void round_keys(uint64_t seed, int i, uint32_t *keys) {
    const uint32_t r = (uint32_t)i >> 1;
    keys[i] = (i & 1) ? (uint32_t)(seed >> 32) + r * 0xBB67AE85u : (uint32_t)seed + r * 0x9E3779B9u;
}
__device__ __forceinline__ uint4 sr_keyed(const uint32_t *keys, uint64_t q, uint32_t stream) {
    uint4 c = make_uint4((uint32_t)q, (uint32_t)(q >> 32), stream, 0u);
#pragma unroll
    for (int r = 0; r < 10; r += 2) {
        const uint4 k = *reinterpret_cast<const uint4 *>(keys + 2 * r);
        uint64_t p0 = (uint64_t)0xD2511F53u * c.x, p1 = (uint64_t)0xCD9E8D57u * c.z;
        c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k.x, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k.y, (uint32_t)p0);
        p0 = (uint64_t)0xD2511F53u * c.x;
        p1 = (uint64_t)0xCD9E8D57u * c.z;
        c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ k.z, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ k.w, (uint32_t)p0);
    }
    return c;
}

// One value with its random byte.
template <int kType> __device__ __forceinline__ uint8_t encode1_sr(float h, float inv, uint32_t byte) {
    if constexpr (kType == SSD_E4M3) {
        const uint32_t f = __half_as_ushort(__float2half_rn(__fmul_rn(h, inv * 0.00390625f)));
        return (uint8_t)((((f & 0x7fffu) + (byte & 0x7fu)) >> 7) | ((f >> 8) & 0x80u));
    } else {
        // floor(h inv + u), u = (byte + 1/2) / 256 (the mantissa of 128 + u, exactly), as
        // the low byte of the sum with 1.5 2^23 rounded down; product and sum each rounded
        const float u = __uint_as_float(0x43000080u | (byte << 8)) - 128.f;
        return (uint8_t)__float_as_uint(__fadd_rd(__fadd_rn(__fmul_rn(h, inv), u), 12582912.f));
    }
}

// Four values with the four random bytes of `word`, packed low to high.
template <int kType> __device__ __forceinline__ uint32_t encode4_sr(const float *h, float inv, uint32_t word) {
    if constexpr (kType == SSD_E4M3) {
        // values 0, 2 and 1, 3 as pairs of fp16, doubled with the random bits
        // doubled: the high byte of each half then holds the seven bits that stay
        // (fp16's top exponent bit is 0 below 2); the sign comes from the fp16
        const float2 s2 = make_float2(inv * 0.00390625f, inv * 0.00390625f);
        const float2 lo = mul2(make_float2(h[0], h[1]), s2), hi = mul2(make_float2(h[2], h[3]), s2);
        const __half2 even = __floats2half2_rn(lo.x, hi.x), odd = __floats2half2_rn(lo.y, hi.y);
        uint32_t fe, fo;
        memcpy(&fe, &even, 4);
        memcpy(&fo, &odd, 4);
        const uint32_t xe = 2u * fe + ((word << 1) & 0x00fe00feu), xo = 2u * fo + ((word >> 7) & 0x00fe00feu);
        return __byte_perm((fe & 0x80008000u) | (xe & 0x7f007f00u), (fo & 0x80008000u) | (xo & 0x7f007f00u), 0x7351);
    } else {
        const float2 inv2 = make_float2(inv, inv);
        const float2 lo = mul2(make_float2(h[0], h[1]), inv2), hi = mul2(make_float2(h[2], h[3]), inv2);
        const float v[4] = {lo.x, lo.y, hi.x, hi.y};
        uint32_t t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = __uint_as_float(__byte_perm(word, 0x43000080u, 0x7604 | (i << 4))) - 128.f;
            t[i] = __float_as_uint(__fadd_rd(__fadd_rn(v[i], u), 12582912.f));
        }
        return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    }
}

// The random bytes of a row of n codes that begins at flat element e0, written
// to `bytes` (16-byte aligned, rand_blocks(n) blocks) by the L lanes that share
// the row; element e0 + i has byte (e0 & 15) + i.  Whole warps call it.
constexpr int rand_blocks(int n) { return (n + 30) / 16; }
template <int L>
__device__ __forceinline__ void row_bytes(uint4 *bytes, const uint32_t *keys, uint64_t e0, int n, int lane) {
    __syncwarp();           // the row before has been read
    const int blocks = ((int)(e0 & 15) + n + 15) >> 4;
    for (int i = lane; i < blocks; i += L) bytes[i] = sr_keyed(keys, (e0 >> 4) + i, 2u);
    __syncwarp();
}

// V values of flat elements e0 .. as codes.  V = 16 is a whole Philox block
// (e0 a multiple of 16); fewer read their bytes at `bytes`, see row_bytes.
template <int kType, int V>
__device__ __forceinline__ Pack<uint8_t, V> encode8_sr(const float *h, float inv, const uint32_t *keys, uint64_t e0,
                                                       const uint8_t *bytes) {
    Pack<uint8_t, V> out;
    if constexpr (V >= 4) {         // e0 is a multiple of V: whole words
        uint32_t word[V / 4], w[V / 4];
        if constexpr (V == 16) {
            const uint4 r = sr_keyed(keys, e0 >> 4, 2u);
            word[0] = r.x;
            word[1] = r.y;
            word[2] = r.z;
            word[3] = r.w;
        } else {
#pragma unroll
            for (int j = 0; j < V / 4; ++j) word[j] = *reinterpret_cast<const uint32_t *>(bytes + 4 * j);
        }
#pragma unroll
        for (int j = 0; j < V; j += 4) w[j / 4] = encode4_sr<kType>(h + j, inv, word[j / 4]);
        memcpy(out.v, w, V);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out.v[j] = encode1_sr<kType>(h[j], inv, bytes[j]);
    }
    return out;
}

// The larger magnitude; NaN if any is NaN.
__device__ __forceinline__ float max_abs(float m, float u, float v) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(u), "f"(v));
    return r;
}

// Largest magnitude and sum over the L lanes that share a row.
template <int L> __device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        const float v = __shfl_xor_sync(0xffffffffu, m, o);
        m = max_abs(m, v, v);
    }
    return m;
}
template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace ssd
