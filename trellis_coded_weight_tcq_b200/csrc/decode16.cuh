// decode16.cuh -- decoding of trellis states to binary16 weights, shared by the
// kernel that writes the matrix out and the product that decodes as it goes.
#pragma once

#include "codes.cuh"

namespace tcq {

// How the codewords are held: the table in shared memory as it came, or none.
enum Code16 { kCode16F32 = 0, kCode16F16 = 1, kCode16Mad = 2 };

__host__ __device__ constexpr size_t table_bytes(int code, int L)
{
    return code == kCode16Mad ? 0 : (((size_t)(code == kCode16F16 ? 2 : 4) << L) + 15) & ~(size_t)15;
}

// Copies the table to shared memory (16-byte asynchronous copies when its address
// allows); the caller synchronises.
template <int CODE>
__device__ __forceinline__ void stage_table(unsigned char* sm, const void* cb, int cb_f16, int L)
{
    if constexpr (CODE != kCode16Mad) {
        const int bytes = (CODE == kCode16F16 ? 2 : 4) << L;
        const unsigned char* src = static_cast<const unsigned char*>(cb);
        if ((reinterpret_cast<uintptr_t>(src) & 15) == 0 && bytes % 16 == 0) {
            const uint32_t dst = (uint32_t)__cvta_generic_to_shared(sm);
            for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i),
                             "l"(src + 16 * (size_t)i) : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            for (int i = threadIdx.x; i < bytes / 2; i += blockDim.x)
                reinterpret_cast<uint16_t*>(sm)[i] = reinterpret_cast<const uint16_t*>(src)[i];
        }
    }
}

// The states of N consecutive weights whose first is weight t0 of its block (N | t0),
// from the two stream words that end with the last window (word -1 is the start
// state).  For N = 8, or 4, and k <= 4 the windows, N k + L - k <= 44 bits, lie in
// those two words.
template <int K, int N>
__device__ __forceinline__ void windows(uint32_t hi, uint32_t lo, int t0, uint32_t mask, uint32_t (&s)[N])
{
    const int down = (32 - ((K * (t0 + N)) & 31)) & 31;  // stream bits behind the last window in lo
    const uint32_t a = __funnelshift_r(lo, hi, down), b = hi >> down;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int sh = (N - 1 - i) * K;
        s[i] = (sh <= 16 ? a >> sh : __funnelshift_r(a, b, sh)) & mask;
    }
}

// Two weights, scale * c[s] rounded to binary16 (the first in the low half).
template <int CODE>
__device__ __forceinline__ uint32_t weight_pair(uint32_t s0, uint32_t s1, const unsigned char* tab, float scale)
{
    float c0, c1;
    if constexpr (CODE == kCode16Mad) {
        c0 = mad_codeword(s0);
        c1 = mad_codeword(s1);
    } else if constexpr (CODE == kCode16F16) {
        c0 = __half2float(reinterpret_cast<const __half*>(tab)[s0]);
        c1 = __half2float(reinterpret_cast<const __half*>(tab)[s1]);
    } else {
        c0 = reinterpret_cast<const float*>(tab)[s0];
        c1 = reinterpret_cast<const float*>(tab)[s1];
    }
    const __half2 h = __floats2half2_rn(c0 * scale, c1 * scale);
    return *reinterpret_cast<const uint32_t*>(&h);
}

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

// 2^e with e held to the normal range.
__device__ __forceinline__ float pow2_clamped(int e)
{
    e = e < -126 ? -126 : e > 127 ? 127 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace tcq
