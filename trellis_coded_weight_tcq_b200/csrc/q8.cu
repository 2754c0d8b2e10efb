// q8.cu -- 8-bit activation checkpoints: packing, unpacking, and the gradient
// through an activation from a packed pre-activation (format: q8.cuh).
//
// All three are bound by memory: 3 + 1/32 bytes per element to pack or unpack, 5 + 1/32
// for the gradient.  4096 x 14336 on a B200 (copies run at 6.4 TB/s): pack 26 us and unpack
// 29 us (178 MB, 6.8 and 6.1 TB/s), gradient with its column sums 58 us (296 MB, 5.1 TB/s;
// the slopes' transcendentals take most of the issue slots beside the loads).
// Rows of a multiple of 8 elements (16 to pack) with 16-byte aligned 16-bit rows move whole
// 16-byte vectors; other shapes take one element per lane, a warp per group, which needs
// no alignment at all (unpacking reads such codes by the byte where its rows out are
// aligned).  Rows that follow one another without gaps and hold whole groups
// are one long row.
#include "gemm.cuh"
#include "pdl.cuh"
#include "q8.cuh"

namespace tcq {

namespace {

constexpr int kThreads = 256;

template <int XT>
__device__ __forceinline__ void load8(const uint16_t* p, float* f)
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
__device__ __forceinline__ void store8(uint16_t* p, const float* f)
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

// Rows of a grid: CTAs take rows blockIdx.x, + gridDim.x, ... and pieces of a row
// blockIdx.y, + gridDim.y, ...

// ---- pack: 16 elements per thread, two neighbouring lanes per group
template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) pack8_vec_kernel(const uint16_t* x, long long ldx, long long n,
                                                             long long cols, uint8_t* codes, uint8_t* scales)
{
    const long long groups = (cols + 31) / 32;
    for (long long r = blockIdx.x; r < n; r += gridDim.x) {
        const uint16_t* xr = x + r * ldx;
        uint8_t* cr = codes + r * cols;
        uint8_t* sr = scales + r * groups;
        // the last group's second lane may hold nothing
        for (long long i = (long long)blockIdx.y * blockDim.x + threadIdx.x; i - (threadIdx.x & 31) < 2 * groups;
             i += (long long)gridDim.y * blockDim.x) {
            const long long c = 16 * i;
            const bool in = c < cols && TCQ_IN_BOUNDS(r * ldx + c + 15, (n - 1) * ldx + cols) &&
                            TCQ_IN_BOUNDS(r * cols + c + 15, n * cols);
            uint32_t w[8] = {};
            if (in) {
                const uint4 a = *reinterpret_cast<const uint4*>(xr + c), b = *reinterpret_cast<const uint4*>(xr + c + 8);
                w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
                w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            }
            // magnitudes order as integers in either 16-bit type, infinities and NaN on top
            uint32_t top = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            const float2 tops = x_unpack2<XT>(top);
            const uint32_t byte = q8_scale_byte<FMT>(max(__float_as_uint(tops.x), __float_as_uint(tops.y)));
            const float inv = q8_inv(byte);
            uint32_t code[4] = {};
            if (byte != 255u) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 p = x_unpack2<XT>(w[2 * j]), q = x_unpack2<XT>(w[2 * j + 1]);
                    const float f[4] = {p.x, p.y, q.x, q.y};
                    code[j] = q8_encode4<FMT>(f, inv);
                }
            }
            if (in) {
                *reinterpret_cast<uint4*>(cr + c) = make_uint4(code[0], code[1], code[2], code[3]);
                if ((i & 1) == 0 && TCQ_IN_BOUNDS(r * groups + i / 2, n * groups)) sr[i / 2] = (uint8_t)byte;
            }
        }
    }
}

template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) pack8_kernel(const uint16_t* x, long long ldx, long long n, long long cols,
                                                         uint8_t* codes, uint8_t* scales)
{
    const long long groups = (cols + 31) / 32;
    for (long long r = blockIdx.x; r < n; r += gridDim.x) {
        for (long long g = (long long)blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32; g < groups;
             g += (long long)gridDim.y * (blockDim.x / 32)) {
            const long long c = 32 * g + (threadIdx.x & 31);
            const float v = c < cols && TCQ_IN_BOUNDS(r * ldx + c, (n - 1) * ldx + cols) ? x_load<XT>(x, r * ldx + c) : 0.f;
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
            const uint32_t byte = q8_scale_byte<FMT>(top);
            const float inv = q8_inv(byte);
            if (c < cols && TCQ_IN_BOUNDS(r * cols + c, n * cols)) codes[r * cols + c] = inv != 0.f ? (uint8_t)q8_encode<FMT>(v, inv) : (uint8_t)0;
            if ((threadIdx.x & 31) == 0 && TCQ_IN_BOUNDS(r * groups + g, n * groups)) scales[r * groups + g] = (uint8_t)byte;
        }
    }
}

// ---- unpack
// Eight elements per thread and step, so that a warp's stores are one run; two steps'
// loads in flight.  BYTES: rows of codes that start anywhere, or do not end on the eighth
// element, read byte by byte (650 x 6210: 15.5 us element by element, 7.8 so).
template <int XT, int FMT, bool BYTES>
__global__ void __launch_bounds__(kThreads) unpack8_vec_kernel(const uint8_t* codes, const uint8_t* scales, long long n,
                                                               long long cols, uint16_t* x, long long ldx)
{
    const long long groups = (cols + 31) / 32, pieces = BYTES ? (cols + 7) / 8 : cols / 8;
    const long long step = blockDim.x;
    pdl_release();  // the weight gradient's next launch
    for (long long r = blockIdx.x; r < n; r += gridDim.x) {
        const uint8_t* cr = codes + r * cols;
        auto fetch = [&](long long i) {
            if constexpr (!BYTES)
                return TCQ_IN_BOUNDS(r * cols + 8 * i + 7, n * cols) ? __ldg(reinterpret_cast<const uint2*>(cr) + i)
                                                                     : make_uint2(0u, 0u);
            uint32_t b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = 8 * i + j < cols && TCQ_IN_BOUNDS(r * cols + 8 * i + j, n * cols) ? __ldg(cr + 8 * i + j) : 0u;
            return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
        };
        const uint8_t* sr = scales + r * groups;
        auto group = [&](long long g) { return TCQ_IN_BOUNDS(r * groups + g, n * groups) ? (uint32_t)__ldg(sr + g) : 0u; };
        uint16_t* xr = x + r * ldx;
        for (long long i = (long long)blockIdx.y * 2 * step + threadIdx.x; i < pieces; i += (long long)gridDim.y * 2 * step) {
            const bool two = i + step < pieces;
            uint2 w[2];
            uint32_t byte[2];
            w[0] = fetch(i);
            byte[0] = group(i / 4);
            if (two) {
                w[1] = fetch(i + step);
                byte[1] = group((i + step) / 4);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && !two) break;
                const float s = q8_scale(byte[h]);
                float f[8];
                q8_codes4<FMT>(w[h].x, f);
                q8_codes4<FMT>(w[h].y, f + 4);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = in_range<XT>(f[j] * s);
                const long long c = 8 * (i + h * step);
                if (BYTES && c + 8 > cols) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < cols && TCQ_IN_BOUNDS(r * ldx + c + j, (n - 1) * ldx + cols)) xr[c + j] = x_bits<XT>(f[j]);
                } else if (TCQ_IN_BOUNDS(r * ldx + c + 7, (n - 1) * ldx + cols)) {
                    store8<XT>(xr + c, f);
                }
            }
        }
    }
}

template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads) unpack8_kernel(const uint8_t* codes, const uint8_t* scales, long long n,
                                                           long long cols, uint16_t* x, long long ldx)
{
    const long long groups = (cols + 31) / 32;
    pdl_release();
    for (long long r = blockIdx.x; r < n; r += gridDim.x) {
        for (long long c = (long long)blockIdx.y * blockDim.x + threadIdx.x; c < cols;
             c += (long long)gridDim.y * blockDim.x)
            if (TCQ_IN_BOUNDS(r * ldx + c, (n - 1) * ldx + cols) && TCQ_IN_BOUNDS(r * cols + c, n * cols) &&
                TCQ_IN_BOUNDS(r * groups + c / 32, n * groups))
                x[r * ldx + c] = x_bits<XT>(
                    in_range<XT>(q8_decode<FMT>(codes[r * cols + c], q8_scale(__ldg(scales + r * groups + c / 32)))));
    }
}

// ---- gradient through the activation
// A CTA owns a strip of columns and a range of rows; its threads keep their columns'
// sums in registers, join the row threads' sums in shared memory, and write one
// partial sum per column and range.  A second kernel adds the ranges in order.
constexpr int kRowThreads = 8;

template <int XT, int FMT, int ACT, int CPT>
__global__ void __launch_bounds__(kThreads, 4) act_grad8_kernel(ActGradArgs a)
{
    __shared__ float part[kRowThreads][32 * CPT + 1];
    const int ct = threadIdx.x & 31, rt = threadIdx.x >> 5;
    const long long c = ((long long)blockIdx.x * 32 + ct) * CPT;
    const long long r0 = a.n * blockIdx.y / gridDim.y, r1 = a.n * (blockIdx.y + 1) / gridDim.y;
    const long long groups = (a.rows + 31) / 32;
    constexpr int P = CPT == 1 ? 1 : CPT / 2;  // pairs of columns
    F2 sum[P];
#pragma unroll
    for (int i = 0; i < P; ++i) sum[i] = f2(0.f, 0.f);
    if (c < a.rows) {
        // a row's loads, one row ahead of their use
        struct Row {
            uint4 d;
            uint2 z;
            uint32_t byte;
        };
        const long long first = r0 + rt;
        int rows = first < r1 ? (int)((r1 - first + kRowThreads - 1) / kRowThreads) : 0, ahead = rows;
        const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + first * a.lddy + c;
        const uint8_t* zc = ACT == TCQ_ACT_NONE ? nullptr : a.z_codes + first * a.rows + c;
        const uint8_t* zs = ACT == TCQ_ACT_NONE ? nullptr : a.z_scales + first * groups + c / 32;
        auto fetch = [&]() {
            Row v = {};
            if (ahead-- > 0 &&
                TCQ_IN_BOUNDS(dy - static_cast<const uint16_t*>(a.dy) + CPT - 1, (a.n - 1) * a.lddy + a.rows)) {
                if constexpr (CPT == 8)
                    v.d = *reinterpret_cast<const uint4*>(dy);
                else
                    v.d.x = *dy;
                dy += kRowThreads * a.lddy;
                if constexpr (ACT != TCQ_ACT_NONE) {
                    if (!TCQ_IN_BOUNDS(zc - a.z_codes + CPT - 1, a.n * a.rows) || !TCQ_IN_BOUNDS(zs - a.z_scales, a.n * groups))
                        return v;
                    if constexpr (CPT == 8)
                        v.z = __ldg(reinterpret_cast<const uint2*>(zc));
                    else
                        v.z.x = __ldg(zc);
                    v.byte = __ldg(zs);
                    zc += kRowThreads * a.rows;
                    zs += kRowThreads * groups;
                }
            }
            return v;
        };
        uint16_t* dz = static_cast<uint16_t*>(a.dz) + first * a.lddz + c;
        Row now = fetch();
        for (; rows > 0; --rows) {
            const Row next = fetch();
            float z[8];
            float s = 0.f;
            if constexpr (ACT != TCQ_ACT_NONE) {
                s = q8_slope_scale<FMT>(now.byte);
                q8_codes4<FMT>(now.z.x, z);
                if constexpr (CPT == 8) q8_codes4<FMT>(now.z.y, z + 4);
            }
            const uint32_t d[4] = {now.d.x, now.d.y, now.d.z, now.d.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 g = x_unpack2<XT>(d[i]);
                F2 t = f2(g.x, g.y);
                if constexpr (ACT != TCQ_ACT_NONE)
                    t = f2_mul(t, act_slope2<ACT>(f2_mul(f2(z[2 * i], z[2 * i + 1]), f2(s, s))));
                sum[i] = f2_add(sum[i], t);
                float u, v;
                f2_split(t, u, v);
                o[i] = x_pack2<XT>(u, v);
            }
            if (TCQ_IN_BOUNDS(dz - static_cast<uint16_t*>(a.dz) + CPT - 1, (a.n - 1) * a.lddz + a.rows)) {
                if constexpr (CPT == 8)
                    *reinterpret_cast<uint4*>(dz) = make_uint4(o[0], o[1], o[2], o[3]);
                else
                    *dz = (uint16_t)o[0];
            }
            dz += kRowThreads * a.lddz;
            now = next;
        }
    }
    if (!a.partial) return;  // the same in every thread
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float u, v;
        f2_split(sum[i], u, v);
        part[rt][ct * CPT + 2 * i] = u;
        if (CPT > 1) part[rt][ct * CPT + 2 * i + 1] = v;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 32 * CPT; j += kThreads) {
        const long long col = (long long)blockIdx.x * 32 * CPT + j;
        if (col >= a.rows) continue;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kRowThreads; ++k) s += part[k][j];
        if (TCQ_IN_BOUNDS((long long)blockIdx.y * a.rows + col, a.splits * a.rows))
            a.partial[(long long)blockIdx.y * a.rows + col] = s;
    }
}

// 32 columns per CTA, the ranges shared among eight threads each, then joined in order.
__global__ void __launch_bounds__(kThreads) sum_ranges_kernel(const float* partial, int ranges, long long rows, float* out)
{
    __shared__ float part[kRowThreads][32];
    pdl_wait();
    const int ct = threadIdx.x & 31, rt = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + ct;
    float s = 0.f;
    if (c < rows) {
#pragma unroll 4
        for (int i = rt; i < ranges && TCQ_IN_BOUNDS((long long)i * rows + c, ranges * rows); i += kRowThreads) s += partial[(long long)i * rows + c];
    }
    part[rt][ct] = s;
    __syncthreads();
    if (rt == 0 && c < rows) {
#pragma unroll
        for (int k = 1; k < kRowThreads; ++k) s += part[k][ct];
        if (TCQ_IN_BOUNDS(c, rows)) out[c] = s;
    }
}

// (rows, columns) of a grid over [n, cols] with `per` columns per thread
dim3 row_grid(long long n, long long cols, int per, int threads, int num_sms)
{
    const long long most = 16ll * num_sms;
    long long y = (cols + (long long)per * threads - 1) / ((long long)per * threads);
    if (y > most) y = most;
    long long x = (most + y - 1) / y;
    if (x > n) x = n;
    return dim3((unsigned)x, (unsigned)y);
}

// threads for rows of `items` items
int row_threads(long long items) { return items >= kThreads ? kThreads : (int)((items + 31) / 32 * 32); }

template <int XT, int FMT>
cudaError_t pack_as(const void* x, long long ldx, long long n, long long cols, uint8_t* codes, uint8_t* scales,
                    int num_sms, cudaStream_t stream)
{
    const uint16_t* xi = static_cast<const uint16_t*>(x);
    if (cols % 32 == 0 && (ldx == cols || n == 1)) {
        cols *= n;
        n = 1;
        ldx = cols;
    }
    if (cols % 16 == 0 && ldx % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(codes)) & 15) == 0) {
        const int threads = row_threads(cols / 16);
        pack8_vec_kernel<XT, FMT><<<row_grid(n, cols, 16, threads, num_sms), threads, 0, stream>>>(xi, ldx, n, cols, codes,
                                                                                                 scales);
    } else {
        const int threads = row_threads(cols);
        pack8_kernel<XT, FMT><<<row_grid(n, cols, 1, threads, num_sms), threads, 0, stream>>>(xi, ldx, n, cols, codes,
                                                                                            scales);
    }
    return cudaGetLastError();
}

template <int XT, int FMT>
cudaError_t unpack_as(const uint8_t* codes, const uint8_t* scales, long long n, long long cols, void* x, long long ldx,
                      int num_sms, cudaStream_t stream)
{
    uint16_t* xo = static_cast<uint16_t*>(x);
    if (cols % 32 == 0 && (ldx == cols || n == 1)) {
        cols *= n;
        n = 1;
        ldx = cols;
    }
    if (ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0) {
        const int threads = row_threads((cols + 7) / 8);
        const bool whole = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(codes) & 7) == 0;
        const auto kernel = whole ? unpack8_vec_kernel<XT, FMT, false> : unpack8_vec_kernel<XT, FMT, true>;
        kernel<<<row_grid(n, cols, 16, threads, num_sms), threads, 0, stream>>>(codes, scales, n, cols, xo, ldx);
    } else {
        const int threads = row_threads(cols);
        unpack8_kernel<XT, FMT><<<row_grid(n, cols, 1, threads, num_sms), threads, 0, stream>>>(codes, scales, n, cols, xo,
                                                                                              ldx);
    }
    return cudaGetLastError();
}

template <int XT, int FMT, int ACT>
void act_grad_launch(const ActGradArgs& a, cudaStream_t stream)
{
    const bool vec = a.rows % 8 == 0 && a.lddy % 8 == 0 && a.lddz % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dz)) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.z_codes) & 7) == 0;
    const dim3 grid((unsigned)((a.rows + (vec ? 255 : 31)) / (vec ? 256 : 32)), (unsigned)a.splits);
    if (vec)
        act_grad8_kernel<XT, FMT, ACT, 8><<<grid, kThreads, 0, stream>>>(a);
    else
        act_grad8_kernel<XT, FMT, ACT, 1><<<grid, kThreads, 0, stream>>>(a);
}

template <int XT, int FMT>
cudaError_t act_grad_as(const ActGradArgs& a, cudaStream_t stream)
{
    switch (a.act) {
    case TCQ_ACT_RELU: act_grad_launch<XT, FMT, TCQ_ACT_RELU>(a, stream); break;
    case TCQ_ACT_SILU: act_grad_launch<XT, FMT, TCQ_ACT_SILU>(a, stream); break;
    case TCQ_ACT_GELU: act_grad_launch<XT, FMT, TCQ_ACT_GELU>(a, stream); break;
    case TCQ_ACT_GELU_TANH: act_grad_launch<XT, FMT, TCQ_ACT_GELU_TANH>(a, stream); break;
    default: act_grad_launch<XT, FMT, TCQ_ACT_NONE>(a, stream); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dbias) return e;
    return launch_pdl(sum_ranges_kernel, dim3((unsigned)((a.rows + 31) / 32)), dim3(kThreads), 0, stream, true,
                      static_cast<const float*>(a.partial), a.splits, a.rows, a.dbias);
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

// Row ranges of the gradient's sums: about 4096 CTAs of 256 columns (several rounds of
// what the SMs hold), at least 32 rows each.  A function of the shape alone, so that
// a sum's order is the same on every device.
int act_grad8_splits(long long n, long long rows)
{
    long long s = 4096 / ((rows + 255) / 256);
    if (s > n / 32) s = n / 32;
    return s < 1 ? 1 : (int)s;
}

cudaError_t launch_act_grad8(const ActGradArgs& a, int xdtype, int format, cudaStream_t stream)
{
    return TCQ_BY_TYPES(act_grad_as, xdtype, format, a, stream);
}

#undef TCQ_BY_TYPES

}  // namespace tcq
