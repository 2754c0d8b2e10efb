// q8.cuh -- the 8-bit activation format and the activation functions, shared by
// the checkpoint kernels and the epilogues of the matrix products.
//
// 32 neighbours of a row share a power-of-two scale 2^e, stored as the byte e + 127
// (0 .. 254); an element is an int8 (|q| <= 127) or an e4m3 number.  e is the least
// exponent with amax <= 127 * 2^e (448 * 2^e), at least -127, so no element
// saturates.  Scaling by a power of two is exact and the rounding to nearest even
// is the only one: an element is off by at most 2^e / 2 (int8), or half a step of
// e4m3, 2^-4 of its value.  A group with an infinity or a NaN has the byte 255 and
// stands for 32 NaNs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace tcq {

constexpr int kQ8Group = 32;

__device__ __forceinline__ float pow2f(int e)  // 2^e, -127 <= e <= 127
{
    return __uint_as_float(e > -127 ? (uint32_t)(e + 127) << 23 : 0x00400000u);
}

// The byte of a group's scale from its largest magnitude's bits (sign cleared;
// 0x7f800000 and above for an infinity or NaN).
template <int FMT>
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return 255u;
    // amax = 1.f * 2^(b - 127) with b its exponent field (0: subnormal, below
    // 2^-126: the least byte 0 holds it).  int8: 127 = 1.984375 * 2^6; e4m3: 448 = 1.75 * 2^8.
    const int b = (int)(amax_bits >> 23);
    const uint32_t f = amax_bits & 0x7fffffu;
    const int e = FMT == TCQ_Q8_INT8 ? b - 6 + (f > 0x7e0000u) : b - 8 + (f > 0x600000u);
    return e > 0 ? (uint32_t)e : 0u;
}

// A code from v with inv = 2^-e of its group.
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode(float v, float inv)
{
    if constexpr (FMT == TCQ_Q8_INT8)
        return (uint32_t)__float2int_rn(v * inv) & 0xffu;
    else
        return (uint32_t)__nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
}

template <int FMT>
__device__ __forceinline__ float q8_decode(uint32_t code, float scale)
{
    if constexpr (FMT == TCQ_Q8_INT8)
        return (float)(int)(signed char)code * scale;
    else
        return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3))) * scale;
}

__device__ __forceinline__ float q8_scale(uint32_t byte)
{
    return byte == 255u ? __int_as_float(0x7fffffff) : pow2f((int)byte - 127);
}

// inv for q8_encode; 0 for a group of NaNs, whose codes are then 0
__device__ __forceinline__ float q8_inv(uint32_t byte) { return byte == 255u ? 0.f : pow2f(127 - (int)byte); }

// ---- 16-bit activations
template <int XT>
__device__ __forceinline__ float x_load(const void* p, long long i)
{
    if constexpr (XT == TCQ_X_BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    else
        return __half2float(reinterpret_cast<const __half*>(p)[i]);
}

// rounds to nearest even
template <int XT>
__device__ __forceinline__ uint16_t x_bits(float v)
{
    if constexpr (XT == TCQ_X_BF16)
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        return __half_as_ushort(__float2half_rn(v));
}

template <int XT>
__device__ __forceinline__ uint32_t x_pack2(float lo, float hi)
{
    if constexpr (XT == TCQ_X_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <int XT>
__device__ __forceinline__ float2 x_unpack2(uint32_t v)
{
    if constexpr (XT == TCQ_X_BF16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// ---- activations.  silu(z) = z / (1 + e^-z); gelu(z) = z (1 + erf(z / sqrt 2)) / 2;
// gelu_tanh(z) = z (1 + tanh u) / 2 = z / (1 + e^-2u), u = sqrt(2 / pi) (z + 0.044715 z^3).
constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + e^-t); the exponential overflows to infinity and the quotient to 0 as they should
__device__ __forceinline__ float sigmoidf(float t) { return __fdividef(1.f, 1.f + __expf(-t)); }

__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
    case TCQ_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case TCQ_ACT_SILU: return z == -INFINITY ? -0.f : z * sigmoidf(z);
    case TCQ_ACT_GELU: return z == -INFINITY ? -0.f : 0.5f * z * (1.f + erff(z * 0.7071067811865476f));
    case TCQ_ACT_GELU_TANH: return z == -INFINITY ? -0.f : z * sigmoidf(2.f * kGeluA * (z + kGeluB * z * z * z));
    default: return z;
    }
}

// The activation's derivative (0 at z = 0 for relu).
__device__ __forceinline__ float act_slope(float z, int act)
{
    switch (act) {
    case TCQ_ACT_RELU: return z > 0.f ? 1.f : (z != z ? z : 0.f);
    case TCQ_ACT_SILU: {
        const float s = sigmoidf(z);
        return s * (1.f + z * (1.f - s));
    }
    case TCQ_ACT_GELU:
        return 0.5f * (1.f + erff(z * 0.7071067811865476f)) + z * __expf(-0.5f * z * z) * 0.3989422804014327f;
    case TCQ_ACT_GELU_TANH: {
        // the slope is 0 or 1 long before +-64, and z^2 below must not overflow
        z = z > 64.f ? 64.f : z < -64.f ? -64.f : z;
        const float s = sigmoidf(2.f * kGeluA * (z + kGeluB * z * z * z));
        return s + z * s * (1.f - s) * (2.f * kGeluA) * (1.f + 3.f * kGeluB * z * z);
    }
    default: return 1.f;
    }
}

}  // namespace tcq
