// Device helpers of the mixer operators: element and vector access, the
// activations, and the storage of state rows (8-bit codes among them).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

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
__device__ __forceinline__ void decode(const Pack<typename Stored<kType>::T, V> &p, float (&out)[V]) {
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

// What a row's largest magnitude (as float bits, sign cleared) makes of its
// scale: inv multiplies the values, scale multiplies the codes.
__device__ __forceinline__ void row_scale(uint32_t max_bits, float limit, float *inv, float *scale) {
    const float m = __uint_as_float(max_bits);
    if (max_bits >= 0x7f800000u) {              // an infinity or a NaN in the row
        *inv = 0.f;
        *scale = __uint_as_float(0x7fffffffu);
    } else if (m < 7.888609052210118e-31f) {    // 2^-100
        *inv = *scale = 0.f;
    } else {
        *inv = __fmul_rn(__frcp_rn(m), limit);
        *scale = __fmul_rn(m, 1.f / limit);
    }
}

// Eight-bit stochastic rounding, the random bytes of elements 16 q .. 16 q + 15.
__device__ __forceinline__ uint4 sr_bytes(uint64_t seed, uint64_t q) { return sr_block(seed, q, 2u); }

// V values times inv as codes, to nearest even.
template <int kType, int V>
__device__ __forceinline__ Pack<uint8_t, V> encode8(const float (&h)[V], float inv) {
    Pack<uint8_t, V> out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float v = __fmul_rn(h[j], inv);
        if constexpr (kType == SSD_E4M3) {
            out.v[j] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
        } else {
            // 1.5 2^23 + v: the sum's rounding is the rounding to an integer
            out.v[j] = (uint8_t)__float_as_uint(__fadd_rn(v, 12582912.f));
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

template <int kType, int V>
__device__ __forceinline__ Pack<uint8_t, V> encode8_sr(const float (&h)[V], float inv, uint64_t seed, uint64_t e0) {
    Pack<uint8_t, V> out;
    uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t e = e0 + (uint64_t)j;
        if (j == 0 || (e & 15) == 0) w = sr_bytes(seed, e >> 4);
        const uint32_t word = sr_word(w, (uint32_t)(e >> 2) & 3u);
        out.v[j] = encode8_sr<kType>(h[j], inv, (word >> (8 * ((uint32_t)e & 3u))) & 0xffu);
    }
    return out;
}

// Largest magnitude over the eight lanes that share a row, as float bits.
__device__ __forceinline__ uint32_t max8(uint32_t m) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace ssd
