// decode16.cuh -- decoding of trellis states to binary16 weights, shared by the
// kernel that writes the matrix out and the product that decodes as it goes.
#pragma once

#include <cuda_bf16.h>

#include "codes.cuh"
#include "powers.cuh"

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

// Stream bits of a word behind the window that ends at stream bit `end`.
__device__ __forceinline__ int bits_behind(int end) { return (32 - (end & 31)) & 31; }

// Bytes of a table entry.
__host__ __device__ constexpr int entry_bytes(int code) { return code == kCode16F32 ? 4 : code == kCode16F16 ? 2 : 1; }

// Weight i of N consecutive ones whose windows end with the two words b:a (the last
// window in a's low bits): the state times the entry size, so that a table look-up
// needs no further shift.  For N = 8, or 4, and k <= 4 the windows, N k + L - k <= 44
// bits, lie in the two words.
template <int K, int N, int CODE>
__device__ __forceinline__ uint32_t window_offset(uint32_t b, uint32_t a, int i, uint32_t mask)
{
    constexpr int up = CODE == kCode16F32 ? 2 : CODE == kCode16F16 ? 1 : 0;
    const int sh = (N - 1 - i) * K - up;
    const uint32_t w = sh < 0 ? a << -sh : sh + up <= 16 ? a >> sh : __funnelshift_r(a, b, sh);
    return w & (mask << up);
}

// The codeword at an offset from window_offset.
template <int CODE>
__device__ __forceinline__ float codeword_at(const unsigned char* tab, uint32_t offset)
{
    if constexpr (CODE == kCode16Mad)
        return mad_codeword(offset);
    else if constexpr (CODE == kCode16F16)
        return __half2float(*reinterpret_cast<const __half*>(tab + offset));
    else
        return *reinterpret_cast<const float*>(tab + offset);
}

// Two weights rounded once to binary16, or to bfloat16 (the first in the low half).
template <bool BF16>
__device__ __forceinline__ uint32_t weight_pair(float a, float b)
{
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// N weights, scale * c[s], in pairs; `down`: stream bits of lo behind the last window.
template <int K, int N, int CODE, bool BF16>
__device__ __forceinline__ void decode_weights(uint32_t hi, uint32_t lo, int down, uint32_t mask,
                                               const unsigned char* tab, float scale, uint32_t* out)
{
    const uint32_t a = __funnelshift_r(lo, hi, down), b = hi >> down;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float c0 = codeword_at<CODE>(tab, window_offset<K, N, CODE>(b, a, i, mask));
        const float c1 = codeword_at<CODE>(tab, window_offset<K, N, CODE>(b, a, i + 1, mask));
        out[i / 2] = weight_pair<BF16>(c0 * scale, c1 * scale);
    }
}

// 64 weights from their 2 K stream words and the word before them, the look-ups of 16
// weights in flight while the 16 before are converted.
template <int K, int CODE>
__device__ __forceinline__ void decode_64(const uint32_t (&words)[2 * K], uint32_t before, uint32_t mask,
                                          const unsigned char* tab, float scale, uint32_t (&out)[32])
{
    float c[2][16];
    auto look_up = [&](int step, float (&f)[16]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int q = 2 * step + h;
            const int e = (8 * K * (q + 1) - 1) >> 5, down = bits_behind(8 * K * (q + 1));
            const uint32_t lo = words[e], hi = e > 0 ? words[e > 0 ? e - 1 : 0] : before;
            const uint32_t a = __funnelshift_r(lo, hi, down), b = hi >> down;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[8 * h + i] = codeword_at<CODE>(tab, window_offset<K, 8, CODE>(b, a, i, mask));
        }
    };
    look_up(0, c[0]);
#pragma unroll
    for (int step = 0; step < 4; ++step) {
        if (step < 3) look_up(step + 1, c[(step + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            out[8 * step + i / 2] = weight_pair<false>(c[step & 1][i] * scale, c[step & 1][i + 1] * scale);
        }
    }
}

}  // namespace tcq
