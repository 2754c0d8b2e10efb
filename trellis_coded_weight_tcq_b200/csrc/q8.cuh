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

// Four codes in one word from v with inv = 2^-e of their group.  int8: adding 1.5 *
// 2^23 rounds the (exact) quotient to nearest even and leaves it in the last byte; no
// conversion instruction (they run at a quarter of the rate).
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode4(const float* v, float inv)
{
    if constexpr (FMT == TCQ_Q8_INT8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(fmaf(v[i], inv, 12582912.f));
        return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}

// One code.
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode(float v, float inv)
{
    if constexpr (FMT == TCQ_Q8_INT8)
        return __float_as_uint(fmaf(v, inv, 12582912.f)) & 0xffu;
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

// Four codes of one word, unscaled.  int8: the byte with its sign bit flipped, placed
// in the last bits of 2^23, is 2^23 + 128 + q; no conversion instruction (they run at
// a quarter of the rate).
template <int FMT>
__device__ __forceinline__ void q8_codes4(uint32_t word, float* f)
{
    if constexpr (FMT == TCQ_Q8_INT8) {
        const uint32_t w = word ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i)) - 8388736.f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (8 * i)), __NV_E4M3);
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h));
            f[i] = t.x;
            f[i + 1] = t.y;
        }
    }
}

__device__ __forceinline__ float q8_scale(uint32_t byte)
{
    return byte == 255u ? __int_as_float(0x7fffffff) : pow2f((int)byte - 127);
}

// The scale of a pre-activation whose only use is an activation's slope: held so that
// far values stay far (a nonzero code at the limit is at least 64, where every slope is
// 0 or 1) and z^2 stays finite.
template <int FMT>
__device__ __forceinline__ float q8_slope_scale(uint32_t byte)
{
    constexpr uint32_t most = FMT == TCQ_Q8_INT8 ? 127 + 6 : 127 + 15;
    return q8_scale(byte == 255u || byte < most ? byte : most);
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

// ---- two fp32 operations in one instruction (each rounds like the scalar one)
struct F2 {
    unsigned long long v;
};

__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void f2_split(F2 p, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}

__device__ __forceinline__ F2 f2_mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 f2_add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + 2^t) of both
__device__ __forceinline__ F2 f2_logistic2(F2 t)
{
    float a, b;
    f2_split(t, a, b);
    const F2 d = f2_add(f2(ex2(a), ex2(b)), f2(1.f, 1.f));
    f2_split(d, a, b);
    return f2(rcp(a), rcp(b));
}

constexpr float kLog2e = 1.4426950408889634f;

// Phi(-a) = erfc(a / sqrt 2) / 2 of two a >= 0, and e = exp(-a^2 / 2): Hastings' rational
// approximation of erf (Abramowitz and Stegun 7.1.26, within 1.5e-7), in packed operations
// (a product with 3211 x 12032 outputs through GELU: 143 us with erff, 79 with it).
__device__ __forceinline__ F2 f2_tail(F2 a, F2& e)
{
    constexpr float p = 0.3275911f * 0.7071067811865476f;
    constexpr float c1 = 0.5f * 0.254829592f, c2 = 0.5f * -0.284496736f, c3 = 0.5f * 1.421413741f,
                    c4 = 0.5f * -1.453152027f, c5 = 0.5f * 1.061405429f;
    float x, y;
    f2_split(f2_fma(a, f2(p, p), f2(1.f, 1.f)), x, y);
    const F2 t = f2(rcp(x), rcp(y));
    f2_split(f2_mul(f2_mul(a, a), f2(-0.5f * kLog2e, -0.5f * kLog2e)), x, y);
    e = f2(ex2(x), ex2(y));
    F2 s = f2_fma(t, f2(c5, c5), f2(c4, c4));
    s = f2_fma(t, s, f2(c3, c3));
    s = f2_fma(t, s, f2(c2, c2));
    s = f2_fma(t, s, f2(c1, c1));
    return f2_mul(f2_mul(t, s), e);
}

// |z|, at most the largest finite number; NaN stays
__device__ __forceinline__ float finite_magnitude_of(float z)
{
    float r;
    asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;" : "=f"(r) : "f"(fabsf(z)));
    return r;
}

// z, or the lowest finite number where it is below (whose product with the logistic
// function's 0 is 0); NaN stays
__device__ __forceinline__ float finite_below(float z)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0fFF7FFFFF;" : "=f"(r) : "f"(z));
    return r;
}

// An activation of two z.
template <int ACT>
__device__ __forceinline__ F2 act_value2(F2 z)
{
    if constexpr (ACT == TCQ_ACT_NONE) {
        return z;
    } else {
        float a, b;
        f2_split(z, a, b);
        if constexpr (ACT == TCQ_ACT_RELU) {
            return f2(a > 0.f ? a : (a != a ? a : 0.f), b > 0.f ? b : (b != b ? b : 0.f));
        } else if constexpr (ACT == TCQ_ACT_GELU) {
            // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
            F2 e;
            const F2 m = f2(finite_magnitude_of(a), finite_magnitude_of(b));
            return f2_fma(f2_mul(m, f2(-1.f, -1.f)), f2_tail(m, e), f2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
        } else {
            z = f2(finite_below(a), finite_below(b));
            if constexpr (ACT == TCQ_ACT_SILU) return f2_mul(z, f2_logistic2(f2_mul(z, f2(-kLog2e, -kLog2e))));
            constexpr float a0 = -2.f * kGeluA * kLog2e, a1 = a0 * kGeluB;
            return f2_mul(z, f2_logistic2(f2_mul(z, f2_fma(f2_mul(z, z), f2(a1, a1), f2(a0, a0)))));
        }
    }
}

// N values at once: the choice is made once.
template <int N>
__device__ __forceinline__ void act_values(float (&v)[N], int act)
{
    auto all = [&](auto one) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if constexpr (N == 1) {
                float unused;
                f2_split(one(f2(v[0], 0.f)), v[0], unused);
            } else {
                f2_split(one(f2(v[i], v[i + 1])), v[i], v[i + 1]);
            }
        }
    };
    switch (act) {
    case TCQ_ACT_RELU: all([](F2 z) { return act_value2<TCQ_ACT_RELU>(z); }); break;
    case TCQ_ACT_SILU: all([](F2 z) { return act_value2<TCQ_ACT_SILU>(z); }); break;
    case TCQ_ACT_GELU: all([](F2 z) { return act_value2<TCQ_ACT_GELU>(z); }); break;
    case TCQ_ACT_GELU_TANH: all([](F2 z) { return act_value2<TCQ_ACT_GELU_TANH>(z); }); break;
    default: break;
    }
}

// An activation's derivative at two finite z below 2^33 (0 at 0 for relu).  With s the
// logistic function: silu' = s + z s (1 - s); gelu_tanh' = s + z s (1 - s) 2 u', s at 2 u.
template <int ACT>
__device__ __forceinline__ F2 act_slope2(F2 z)
{
    if constexpr (ACT == TCQ_ACT_SILU) {
        const F2 s = f2_logistic2(f2_mul(z, f2(-kLog2e, -kLog2e)));
        const F2 m = f2_fma(f2_mul(s, f2(-1.f, -1.f)), s, s);
        return f2_fma(m, z, s);
    } else if constexpr (ACT == TCQ_ACT_GELU_TANH) {
        constexpr float a0 = -2.f * kGeluA * kLog2e, a1 = a0 * kGeluB, b0 = 2.f * kGeluA, b1 = 3.f * b0 * kGeluB;
        const F2 zz = f2_mul(z, z);
        const F2 s = f2_logistic2(f2_mul(z, f2_fma(zz, f2(a1, a1), f2(a0, a0))));
        const F2 m = f2_fma(f2_mul(s, f2(-1.f, -1.f)), s, s);
        return f2_fma(m, f2_mul(z, f2_fma(zz, f2(b1, b1), f2(b0, b0))), s);
    } else {
        float a, b;
        f2_split(z, a, b);
        if constexpr (ACT == TCQ_ACT_RELU) {
            return f2(a > 0.f ? 1.f : (a != a ? a : 0.f), b > 0.f ? 1.f : (b != b ? b : 0.f));
        } else {
            F2 e;
            float u, v;
            f2_split(f2_tail(f2(fabsf(a), fabsf(b)), e), u, v);
            const F2 phi = f2(a > 0.f ? 1.f - u : u, b > 0.f ? 1.f - v : v);
            return f2_fma(f2_mul(z, e), f2(0.3989422804014327f, 0.3989422804014327f), phi);
        }
    }
}

}  // namespace tcq
