// q8.cu -- 8-bit activation checkpoints: packing, unpacking, and the gradient
// through an activation from a packed pre-activation (format: q8.cuh).
//
// All three are bound by memory: 3 + 1/32 bytes per element to pack or unpack, 5 + 1/32
// for the gradient.  Rows of a multiple of 8 elements with 16-byte aligned 16-bit
// rows move 8 elements per thread (16- and 8-byte accesses), four neighbouring lanes
// sharing a group; other shapes take one element per lane, a warp per group, which
// needs no alignment at all.
#include "gemm.cuh"
#include "q8.cuh"

namespace tcq {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t max3(uint32_t a, uint32_t b, uint32_t c) { return max(a, max(b, c)); }

// the codes of eight elements
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv)
{
    uint32_t c[2] = {0u, 0u};
    if (inv != 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i / 4] |= q8_encode<FMT>(f[i], inv) << (8 * (i & 3));
    }
    return make_uint2(c[0], c[1]);
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 codes, float scale, float (&f)[8])
{
    const uint32_t c[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = q8_decode<FMT>((c[i / 4] >> (8 * (i & 3))) & 0xffu, scale);
}

template <int XT>
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8])
{
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 t = x_unpack2<XT>(w[h]);
        f[2 * h] = t.x;
        f[2 * h + 1] = t.y;
    }
}

template <int XT>
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(x_pack2<XT>(f[0], f[1]), x_pack2<XT>(f[2], f[3]),
                                              x_pack2<XT>(f[4], f[5]), x_pack2<XT>(f[6], f[7]));
}

// binary16 cannot hold every checkpoint: its largest number stands for what is above
template <int XT>
__device__ __forceinline__ float in_range(float v)
{
    if constexpr (XT == TCQ_X_F16) return v > 65504.f ? 65504.f : v < -65504.f ? -65504.f : v;
    return v;
}

// ---- pack
template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) pack8_vec_kernel(const uint16_t* x, long long ldx, long long n, int cols,
                                                             int groups, uint8_t* codes, uint8_t* scales)
{
    // four lanes per group; the last group's lanes behind the row's end hold nothing
    const int per_row = 4 * groups;
    const long long total = n * per_row;
    const long long stride = (long long)gridDim.x * kThreads;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i - threadIdx.x % 32 < total; i += stride) {
        const long long r = i / per_row;
        const int c = (int)(i - r * per_row) * 8;
        const bool in = i < total && c < cols;
        float f[8] = {};
        uint32_t top = 0u;
        if (in) {
            load8<XT>(x + r * ldx + c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (in) {
            const uint32_t byte = q8_scale_byte<FMT>(top);
            *reinterpret_cast<uint2*>(codes + r * cols + c) = encode8<FMT>(f, q8_inv(byte));
            if ((c & 31) == 0) scales[r * groups + c / 32] = (uint8_t)byte;
        }
    }
}

template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) pack8_kernel(const uint16_t* x, long long ldx, long long n, int cols,
                                                         int groups, uint8_t* codes, uint8_t* scales)
{
    const int lane = threadIdx.x & 31;
    const long long total = n * groups, stride = (long long)gridDim.x * (kThreads / 32);
    for (long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5; i < total; i += stride) {
        const long long r = i / groups;
        const int g = (int)(i - r * groups), c = 32 * g + lane;
        const float v = c < cols ? x_load<XT>(x, r * ldx + c) : 0.f;
        uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
        const uint32_t byte = q8_scale_byte<FMT>(top);
        const float inv = q8_inv(byte);
        if (c < cols) codes[r * cols + c] = inv != 0.f ? (uint8_t)q8_encode<FMT>(v, inv) : (uint8_t)0;
        if (lane == 0) scales[i] = (uint8_t)byte;
    }
}

// ---- unpack
template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) unpack8_vec_kernel(const uint8_t* codes, const uint8_t* scales, long long n,
                                                               int cols, int groups, uint16_t* x, long long ldx)
{
    const int per_row = cols / 8;
    const long long total = n * per_row;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kThreads) {
        const long long r = i / per_row;
        const int c = (int)(i - r * per_row) * 8;
        float f[8];
        decode8<FMT>(*reinterpret_cast<const uint2*>(codes + r * cols + c), q8_scale(scales[r * groups + c / 32]), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = in_range<XT>(f[j]);
        store8<XT>(x + r * ldx + c, f);
    }
}

template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) unpack8_kernel(const uint8_t* codes, const uint8_t* scales, long long n,
                                                           int cols, int groups, uint16_t* x, long long ldx)
{
    const int lane = threadIdx.x & 31;
    const long long total = n * groups, stride = (long long)gridDim.x * (kThreads / 32);
    for (long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5; i < total; i += stride) {
        const long long r = i / groups;
        const int g = (int)(i - r * groups), c = 32 * g + lane;
        if (c < cols)
            x[r * ldx + c] = x_bits<XT>(in_range<XT>(q8_decode<FMT>(codes[r * cols + c], q8_scale(scales[i]))));
    }
}

// ---- gradient through the activation
// A CTA owns a strip of columns and a range of rows; its threads keep their columns'
// sums in registers, join the row threads' sums in shared memory, and write one
// partial sum per column and range.  A second kernel adds the ranges in order.
constexpr int kRowThreads = 8;

template <int XT, int FMT, int CPT>
__global__ void __launch_bounds__(kThreads) act_grad8_kernel(ActGradArgs a, int groups)
{
    __shared__ float part[kRowThreads][32 * CPT + 1];
    const int ct = threadIdx.x & 31, rt = threadIdx.x >> 5;
    const long long c = ((long long)blockIdx.x * 32 + ct) * CPT;
    const long long r0 = a.n * blockIdx.y / gridDim.y, r1 = a.n * (blockIdx.y + 1) / gridDim.y;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
    uint16_t* dz = static_cast<uint16_t*>(a.dz);
    float sum[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) sum[i] = 0.f;
    if (c < a.rows) {
#pragma unroll 2
        for (long long r = r0 + rt; r < r1; r += kRowThreads) {
            float g[CPT], z[CPT];
            if constexpr (CPT == 8) {
                load8<XT>(dy + r * a.lddy + c, g);
                if (a.act != TCQ_ACT_NONE)
                    decode8<FMT>(*reinterpret_cast<const uint2*>(a.z_codes + r * a.rows + c),
                                 q8_scale(a.z_scales[r * groups + c / 32]), z);
            } else {
                g[0] = x_load<XT>(dy, r * a.lddy + c);
                if (a.act != TCQ_ACT_NONE)
                    z[0] = q8_decode<FMT>(a.z_codes[r * a.rows + c], q8_scale(a.z_scales[r * groups + c / 32]));
            }
            switch (a.act) {
            case TCQ_ACT_RELU:
#pragma unroll
                for (int i = 0; i < CPT; ++i) g[i] *= act_slope(z[i], TCQ_ACT_RELU);
                break;
            case TCQ_ACT_SILU:
#pragma unroll
                for (int i = 0; i < CPT; ++i) g[i] *= act_slope(z[i], TCQ_ACT_SILU);
                break;
            case TCQ_ACT_GELU:
#pragma unroll
                for (int i = 0; i < CPT; ++i) g[i] *= act_slope(z[i], TCQ_ACT_GELU);
                break;
            case TCQ_ACT_GELU_TANH:
#pragma unroll
                for (int i = 0; i < CPT; ++i) g[i] *= act_slope(z[i], TCQ_ACT_GELU_TANH);
                break;
            default: break;
            }
#pragma unroll
            for (int i = 0; i < CPT; ++i) sum[i] += g[i];
            if constexpr (CPT == 8)
                store8<XT>(dz + r * a.lddz + c, g);
            else
                dz[r * a.lddz + c] = x_bits<XT>(g[0]);
        }
    }
    if (!a.partial) return;  // the same in every thread
#pragma unroll
    for (int i = 0; i < CPT; ++i) part[rt][ct * CPT + i] = sum[i];
    __syncthreads();
    for (int j = threadIdx.x; j < 32 * CPT; j += kThreads) {
        const long long col = (long long)blockIdx.x * 32 * CPT + j;
        if (col >= a.rows) continue;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kRowThreads; ++k) s += part[k][j];
        a.partial[(long long)blockIdx.y * a.rows + col] = s;
    }
}

__global__ void __launch_bounds__(kThreads) sum_ranges_kernel(const float* partial, int ranges, long long rows, float* out)
{
    const long long c = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (c >= rows) return;
    float s = 0.f;
    for (int i = 0; i < ranges; ++i) s += partial[i * rows + c];
    out[c] = s;
}

template <int XT, int FMT>
cudaError_t pack_as(const void* x, long long ldx, long long n, long long cols, uint8_t* codes, uint8_t* scales,
                    int num_sms, cudaStream_t stream)
{
    const uint16_t* xi = static_cast<const uint16_t*>(x);
    const int groups = (int)((cols + 31) / 32);
    const bool vec = cols % 8 == 0 && ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
    long long grid = (n * groups * (vec ? 4 : 32) + kThreads - 1) / kThreads;
    if (grid > 32ll * num_sms) grid = 32ll * num_sms;
    if (vec)
        pack8_vec_kernel<XT, FMT><<<(int)grid, kThreads, 0, stream>>>(xi, ldx, n, (int)cols, groups, codes, scales);
    else
        pack8_kernel<XT, FMT><<<(int)grid, kThreads, 0, stream>>>(xi, ldx, n, (int)cols, groups, codes, scales);
    return cudaGetLastError();
}

template <int XT, int FMT>
cudaError_t unpack_as(const uint8_t* codes, const uint8_t* scales, long long n, long long cols, void* x, long long ldx,
                      int num_sms, cudaStream_t stream)
{
    uint16_t* xo = static_cast<uint16_t*>(x);
    const int groups = (int)((cols + 31) / 32);
    const bool vec = cols % 8 == 0 && ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
    long long grid = (n * groups * (vec ? 4 : 32) + kThreads - 1) / kThreads;
    if (grid > 32ll * num_sms) grid = 32ll * num_sms;
    if (vec)
        unpack8_vec_kernel<XT, FMT><<<(int)grid, kThreads, 0, stream>>>(codes, scales, n, (int)cols, groups, xo, ldx);
    else
        unpack8_kernel<XT, FMT><<<(int)grid, kThreads, 0, stream>>>(codes, scales, n, (int)cols, groups, xo, ldx);
    return cudaGetLastError();
}

template <int XT, int FMT>
cudaError_t act_grad_as(const ActGradArgs& a, cudaStream_t stream)
{
    const int groups = (int)((a.rows + 31) / 32);
    const bool vec = a.rows % 8 == 0 && a.lddy % 8 == 0 && a.lddz % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dz)) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.z_codes) & 7) == 0;
    const dim3 grid((unsigned)((a.rows + (vec ? 255 : 31)) / (vec ? 256 : 32)), (unsigned)a.splits);
    if (vec)
        act_grad8_kernel<XT, FMT, 8><<<grid, kThreads, 0, stream>>>(a, groups);
    else
        act_grad8_kernel<XT, FMT, 1><<<grid, kThreads, 0, stream>>>(a, groups);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dbias) return e;
    sum_ranges_kernel<<<(unsigned)((a.rows + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a.partial, a.splits,
                                                                                              a.rows, a.dbias);
    return cudaGetLastError();
}

}  // namespace

#define TCQ_BY_TYPES(fn, xt, fmt, ...)                                                                        \
    ((xt) == TCQ_X_BF16 ? ((fmt) == TCQ_Q8_INT8 ? fn<TCQ_X_BF16, TCQ_Q8_INT8>(__VA_ARGS__)                     \
                                                : fn<TCQ_X_BF16, TCQ_Q8_E4M3>(__VA_ARGS__))                    \
                        : ((fmt) == TCQ_Q8_INT8 ? fn<TCQ_X_F16, TCQ_Q8_INT8>(__VA_ARGS__)                      \
                                                : fn<TCQ_X_F16, TCQ_Q8_E4M3>(__VA_ARGS__)))

cudaError_t launch_pack8(const void* x, int xdtype, long long ldx, long long n, long long cols, int format,
                         uint8_t* codes, uint8_t* scales, int num_sms, cudaStream_t stream)
{
    return TCQ_BY_TYPES(pack_as, xdtype, format, x, ldx, n, cols, codes, scales, num_sms, stream);
}

cudaError_t launch_unpack8(const uint8_t* codes, const uint8_t* scales, int format, long long n, long long cols,
                           void* x, int xdtype, long long ldx, int num_sms, cudaStream_t stream)
{
    return TCQ_BY_TYPES(unpack_as, xdtype, format, codes, scales, n, cols, x, ldx, num_sms, stream);
}

// Row ranges of the gradient's sums: about 1024 CTAs of 256 columns (so that every
// SM holds several), at least 32 rows each.  A function of the shape alone, so that
// a sum's order is the same on every device.
int act_grad8_splits(long long n, long long rows)
{
    long long s = 1024 / ((rows + 255) / 256);
    if (s > n / 32) s = n / 32;
    return s < 1 ? 1 : (int)s;
}

cudaError_t launch_act_grad8(const ActGradArgs& a, int xdtype, int format, cudaStream_t stream)
{
    return TCQ_BY_TYPES(act_grad_as, xdtype, format, a, stream);
}

#undef TCQ_BY_TYPES

}  // namespace tcq
