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

// V consecutive elements moved together (one instruction up to 16 bytes).
template <typename T, int V> struct alignas(sizeof(T) * V <= 16 ? sizeof(T) * V : 16) Pack { T v[V]; };

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T *src) {
    return *reinterpret_cast<const Pack<T, V> *>(src);
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T *dst, const Pack<T, V> &p) {
    *reinterpret_cast<Pack<T, V> *>(dst) = p;
}

// v sigmoid(v).  ex2 and rcp approximations: about 2^-21 relative error.
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// softplus(z) = log(1 + e^z) in the overflow-safe form max(z,0) + log1p(e^-|z|)
__device__ __forceinline__ float softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// Two fp32 operations in one instruction, each rounded as by itself.
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

// Stored values as floats; 8-bit codes without their scale.
template <int kType, int V>
__device__ __forceinline__ void decode(const Pack<typename Stored<kType>::T, V> &p, float *out) {
    if constexpr (kType == SSD_E4M3 && V >= 2) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const __half2_raw two =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(p.v[j] | p.v[j + 1] << 8), __NV_E4M3);
            const float2 f = __half22float2(__half2(two));
            out[j] = f.x;
            out[j + 1] = f.y;
        }
    } else if constexpr (kType == SSD_I8 && V >= 4) {
        // the code + 128 as the low byte of 2^23's mantissa
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            uint32_t w;
            memcpy(&w, p.v + j, 4);
            w ^= 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[j + i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | i)) - 8388736.f;
        }
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

// What a row's largest magnitude makes of its scale: inv multiplies the
// values, scale multiplies the codes.
__device__ __forceinline__ void row_scale(float m, float limit, float *inv, float *scale) {
    *inv = __fmul_rn(__frcp_rn(m), limit);
    *scale = __fmul_rn(m, 1.f / limit);
    if (!(m < __int_as_float(0x7f800000))) {    // an infinity or a NaN in the row
        *inv = 0.f;
        *scale = __int_as_float(0x7fffffff);
    } else if (m < 7.888609052210118e-31f) {    // 2^-100
        *inv = *scale = 0.f;
    }
}

// sr_f16 with the dropped bits as an integer where fp16 is normal: there
// (|v| - |lo|) / spacing is the 13 dropped bits over 2^13.
__device__ __forceinline__ __half sr_f16_fast(float v, uint32_t r) {
    const uint32_t bits = __float_as_uint(v), a = bits & 0x7fffffffu;
    if (a < 0x38800000u || a >= 0x47800000u) return sr_f16(v, r);       // below 2^-14, from 2^16 on, inf, NaN
    const uint32_t h = ((a - 0x38000000u) >> 13) + ((a << 19) > r ? 1u : 0u);
    return __ushort_as_half((unsigned short)(h | (bits >> 16 & 0x8000u)));
}

// Eight-bit stochastic rounding, the random bytes of elements 16 q .. 16 q + 15.
__device__ __forceinline__ uint4 sr_bytes(uint64_t seed, uint64_t q) { return sr_block(seed, q, 2u); }

// V values times inv as codes, to nearest even.
template <int kType, int V>
__device__ __forceinline__ Pack<uint8_t, V> encode8(const float *h, float inv) {
    Pack<uint8_t, V> out;
    if constexpr (kType == SSD_E4M3 && V >= 2) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(h[j], inv), __fmul_rn(h[j + 1], inv)), __NV_SATFINITE, __NV_E4M3);
            out.v[j] = (uint8_t)two;
            out.v[j + 1] = (uint8_t)(two >> 8);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float v = __fmul_rn(h[j], inv);
            // int8: 1.5 2^23 + v, whose rounding is the rounding to an integer
            out.v[j] = kType == SSD_E4M3 ? (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3)
                                         : (uint8_t)__float_as_uint(__fadd_rn(v, 12582912.f));
        }
    }
    return out;
}

// The same with random bytes: stochastic rounding, see SSD_E4M3 in ssd_mixer.h.
template <int kType>
__device__ __forceinline__ uint8_t encode8_sr(float h, float inv, uint32_t byte) {
    if constexpr (kType == SSD_E4M3) {
        const uint32_t f = __half_as_ushort(__float2half_rn(__fmul_rn(h, inv) * 0.00390625f));
        return (uint8_t)((((f & 0x7fffu) + (byte & 0x7fu)) >> 7) | ((f >> 8) & 0x80u));
    } else {
        // floor(h inv + u), u = (byte + 1/2) / 256 (the mantissa of 128 + u, exactly), as
        // the low byte of the sum with 1.5 2^23 rounded down
        const float u = __uint_as_float(0x43000080u | (byte << 8)) - 128.f;
        return (uint8_t)__float_as_uint(__fadd_rd(__fmaf_rn(h, inv, u), 12582912.f));
    }
}

// Four values with the four random bytes of `word`, packed low to high.
template <int kType>
__device__ __forceinline__ uint32_t encode8_sr4(const float *h, float inv, uint32_t word) {
    if constexpr (kType == SSD_E4M3) {
        // two fp16 at a time; after the sum and a shift left by one, the high
        // byte of each half holds the seven bits that stay (fp16's top exponent
        // bit is 0 below 2), its sign comes from the unshifted word
        const float s = inv * 0.00390625f;
        const uint32_t r = word & 0x7f7f7f7fu;
        uint32_t x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2 two = __floats2half2_rn(__fmul_rn(h[2 * i], s), __fmul_rn(h[2 * i + 1], s));
            uint32_t f;
            memcpy(&f, &two, 4);
            f += __byte_perm(r, 0u, i ? 0x4342 : 0x4140);
            x[i] = (f & 0x80008000u) | ((f << 1) & 0x7fff7fffu);
        }
        return __byte_perm(x[0], x[1], 0x7531);
    } else {
        uint32_t t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // 128 + byte / 256 + 1/512
            const float u = __uint_as_float(__byte_perm(word, 0x43000080u, 0x7604 | (i << 4))) - 128.f;
            t[i] = __float_as_uint(__fadd_rd(__fmaf_rn(h[i], inv, u), 12582912.f));
        }
        return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    }
}

template <int kType, int V>
__device__ __forceinline__ Pack<uint8_t, V> encode8_sr(const float *h, float inv, uint64_t seed, uint64_t e0) {
    Pack<uint8_t, V> out;
    if constexpr (V >= 4) {         // e0 is a multiple of V: whole words
        const uint4 w = sr_bytes(seed, e0 >> 4);
        uint32_t word[4] = {w.x, w.y, w.z, w.w};
        if constexpr (V == 8) {
            word[0] = (e0 & 8) ? w.z : w.x;
            word[1] = (e0 & 8) ? w.w : w.y;
        } else if constexpr (V == 4) {
            word[0] = sr_word(w, (uint32_t)(e0 >> 2) & 3u);
        }
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const uint32_t c = encode8_sr4<kType>(h + j, inv, word[j / 4]);
            memcpy(out.v + j, &c, 4);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint64_t e = e0 + (uint64_t)j;
            const uint32_t word = sr_word(sr_bytes(seed, e >> 4), (uint32_t)(e >> 2) & 3u);
            out.v[j] = encode8_sr<kType>(h[j], inv, (word >> (8 * ((uint32_t)e & 3u))) & 0xffu);
        }
    }
    return out;
}

// The larger magnitude; NaN if either is NaN.
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

// Largest magnitude over the eight lanes that share a row (NaN if any is).
__device__ __forceinline__ float max8(float m) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace ssd
