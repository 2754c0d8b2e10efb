// powers.cuh -- the powers of two that bring the operands of the binary16 products into
// binary16's range, and their use in the epilogues.
//
// A weight is scale * codeword.  It is stored over the product of two powers, one per row
// of the matrix (the least above its largest finite |scale|) and, for tables, one of the
// table (so that its largest finite entry ends in [2^14, 2^15); the computed code's is
// 2^-14, part of the rows'); the epilogue multiplies both back.  Neither changes a rounding.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tcq {

// Bits of |v|, or 0 for an infinity or NaN (magnitudes then compare as integers).
__device__ __forceinline__ uint32_t finite_magnitude(float v)
{
    const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// The least p with |v| < 2^p, from the bits of |v| (0 for v = 0, -126 for subnormals).
__device__ __forceinline__ int power_above(uint32_t magnitude)
{
    if (magnitude == 0u) return 0;
    const int p = (int)(magnitude >> 23) - 126;
    return p;
}

// 2^e with e held to -126 .. 126, so that its inverse is a normal number too.
__device__ __forceinline__ float pow2_clamped(int e)
{
    e = e < -126 ? -126 : e > 126 ? 126 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The inverse of such a power.
__device__ __forceinline__ float inverse_pow2(float p) { return __uint_as_float(0x7f000000u - __float_as_uint(p)); }

__device__ __forceinline__ int exponent_of(float power) { return (int)(__float_as_uint(power) >> 23) - 127; }

// The product of two powers, held like each of them.
__device__ __forceinline__ float power_product(float a, float b) { return pow2_clamped(exponent_of(a) + exponent_of(b)); }

// 2^e, -252 <= e <= 252, as two factors: v * x * y passes through no number beyond fp32's
// range unless its result is one.
__device__ __forceinline__ float2 power_halves(int e)
{
    const int h = e >> 1;
    return make_float2(__uint_as_float((uint32_t)(h + 127) << 23), __uint_as_float((uint32_t)(e - h + 127) << 23));
}

// A table's power from its largest finite magnitude's bits: the largest entry over it is
// in [2^14, 2^15).
__device__ __forceinline__ float power_of_top(uint32_t top) { return top == 0u ? 1.f : pow2_clamped(power_above(top) - 15); }

// The same from the largest finite magnitudes of the table's parts, one per CTA that
// reads it ahead of the products.
constexpr int kTableParts = 8;

struct TableParts {
    uint4 a, b;
    __device__ __forceinline__ explicit TableParts(const uint32_t* top)
    {
        a = b = make_uint4(0u, 0u, 0u, 0u);
        if (top) {
            a = __ldcg(reinterpret_cast<const uint4*>(top));
            b = __ldcg(reinterpret_cast<const uint4*>(top) + 1);
        }
    }
    __device__ __forceinline__ float power() const
    {
        return power_of_top(max(max(max(a.x, a.y), max(a.z, a.w)), max(max(b.x, b.y), max(b.z, b.w))));
    }
};

__device__ __forceinline__ float table_power(const uint32_t* top) { return TableParts(top).power(); }

// The same from a binary32 table in shared memory, by all threads of a CTA; `warps` a
// word per warp.  `out` (kTableParts words, or nullptr): where the first CTA leaves it
// for table_power.
__device__ __forceinline__ float staged_table_power(const float* table, int entries, uint32_t* warps, uint32_t* out)
{
    uint32_t top = 0u;
    for (int i = threadIdx.x; i < entries; i += blockDim.x) top = max(top, finite_magnitude(table[i]));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = top;
    __syncthreads();
    top = 0u;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) top = max(top, warps[i]);
    if (out && blockIdx.x == 0 && threadIdx.x < kTableParts) out[threadIdx.x] = threadIdx.x == 0 ? top : 0u;
    return power_of_top(top);
}

}  // namespace tcq
