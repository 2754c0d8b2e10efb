// operands.cu -- the passes that bring the activations of a product to binary16 rows,
// and the powers of two of a coded matrix's rows and of its table.
//
// A row's largest element is brought to [2^14, 2^15).  A bfloat16 row is then exact down to
// 2^-31 of that element (eight bits from 2^-17 up end above 2^-24, binary16's last), a
// binary16 one down to 2^-28, and smaller elements are off by at most 2^-25; binary16
// keeps the weights exact where bfloat16 would not.  The rows are read twice (the second time from L2) and written
// once: bound by memory, about 4 bytes per element.
#include "decode16.cuh"
#include "gemm.cuh"
#include "pdl.cuh"
#include "q8.cuh"

namespace tcq {

namespace {

constexpr int kThreads = 256;

// A row's power, from the largest finite |scale| of a row of W: one warp per row.
__device__ __forceinline__ void row_power(const RowPowers& p, long long r)
{
    uint32_t top = 0u;
    for (int j = threadIdx.x & 31; j < p.per_row && TCQ_IN_BOUNDS(r * p.per_row + j, p.rows * p.per_row); j += 32)
        top = max(top, finite_magnitude(__ldg(p.scale + r * p.per_row + j)));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0 && TCQ_IN_BOUNDS(r, p.rows)) {
        const float v = pow2_clamped(power_above(top) - p.down);
        p.out[r] = v;
        if (p.exponents) p.exponents[r] = (uint8_t)(__float_as_uint(v) >> 23);
    }
}

// The largest finite magnitude of a part of the table, 16 bytes a thread and step where
// its address allows (a 128 KB table: four loads in flight per thread of each of the parts).
__device__ __forceinline__ void table_part(const RowPowers& p, int part)
{
    __shared__ uint32_t warps[kThreads / 32];
    const int entries = 1 << p.table_log2, bytes = entries * (p.table_f16 ? 2 : 4);
    const int first = part * kThreads + threadIdx.x;
    uint32_t top = 0u;
    if ((reinterpret_cast<uintptr_t>(p.table) & 15) == 0 && bytes % 16 == 0) {
#pragma unroll 4
        for (int i = first; i < bytes / 16 && TCQ_IN_BOUNDS(16 * i + 15, bytes); i += kTableParts * kThreads) {
            const uint4 v = __ldg(static_cast<const uint4*>(p.table) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float2 t = p.table_f16 ? x_unpack2<TCQ_X_F16>(w[h]) : make_float2(__uint_as_float(w[h]), 0.f);
                top = max(top, max(finite_magnitude(t.x), finite_magnitude(t.y)));
            }
        }
    } else {
#pragma unroll 4
        for (int i = first; i < entries && TCQ_IN_BOUNDS(i, entries); i += kTableParts * kThreads)
            top = max(top, finite_magnitude(load_codeword(p.table, p.table_f16, (uint32_t)i)));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) top = max(top, warps[i]);
        if (TCQ_IN_BOUNDS(part, kTableParts)) p.table_top[part] = top;
    }
}

// The power of two with this exponent field.
__device__ __forceinline__ float power_of(uint32_t exponent) { return __uint_as_float(exponent << 23); }

// One CTA per row: the row's largest finite magnitude, then the row over the power of
// two that brings it to [2^14, 2^15).
template <int XT>
__device__ __forceinline__ void scale_row(const ScaleRows& a, long long r)
{
    __shared__ uint32_t part[kThreads / 32];
    const uint16_t* xr = static_cast<const uint16_t*>(a.x) + r * a.ldx;
    uint16_t* o = static_cast<uint16_t*>(a.out) + r * a.ldo;
    uint32_t top = 0u;
    // the columns' exponent fields with the table's power, held like power_product
    const int table = exponent_of(table_power(a.table_top));
    auto column = [&](uint32_t field) { return power_of((uint32_t)max(min((int)field + table, 253), 1)); };
    auto eight = [&](long long c, float (&f)[8]) {
        const uint4 v = TCQ_IN_BOUNDS(r * a.ldx + c + 7, (a.n - 1) * a.ldx + a.cols) ? *reinterpret_cast<const uint4*>(xr + c)
                                                                                    : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float2 t = x_unpack2<XT>(w[h]);
            f[2 * h] = t.x;
            f[2 * h + 1] = t.y;
        }
        if (a.col_exponents) {  // bytes: as fp32 powers they would be twice the row's own traffic
            const uint2 e = *reinterpret_cast<const uint2*>(a.col_exponents + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] *= column((e.x >> (8 * i)) & 0xffu);
                f[4 + i] *= column((e.y >> (8 * i)) & 0xffu);
            }
        }
    };
    const long long vcols = a.vec ? a.cols / 8 * 8 : 0;
    for (long long c = 8ll * threadIdx.x; c < vcols; c += 8 * kThreads) {
        float f[8];
        eight(c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, finite_magnitude(f[i]));
    }
    for (long long c = vcols + threadIdx.x; c < a.cols && TCQ_IN_BOUNDS(r * a.ldx + c, (a.n - 1) * a.ldx + a.cols); c += kThreads)
        top = max(top, finite_magnitude(x_load<XT>(xr, c) * (a.col_exponents ? column(a.col_exponents[c]) : 1.f)));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, part[i]);
    // |x| < 2^p; the factor stays in the normal range, so tiny rows end lower than 2^15
    int p = 0;
    if (top != 0u) p = power_above(top) - 15;
    if (p < -126) p = -126;
    const float inv = pow2_clamped(-p);
    if (threadIdx.x == 0 && TCQ_IN_BOUNDS(r, a.n)) a.row_pow2[r] = pow2_clamped(p);
    for (long long c = 8ll * threadIdx.x; c < vcols; c += 8 * kThreads) {
        float f[8];
        eight(c, f);
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) w[h] = x_pack2<TCQ_X_F16>(f[2 * h] * inv, f[2 * h + 1] * inv);
        if (TCQ_IN_BOUNDS(r * a.ldo + c + 7, a.n * a.ldo))
            *reinterpret_cast<uint4*>(o + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (long long c = vcols + threadIdx.x; c < a.cols && TCQ_IN_BOUNDS(r * a.ldo + c, a.n * a.ldo); c += kThreads)
        o[c] = x_bits<TCQ_X_F16>(x_load<XT>(xr, c) * (a.col_exponents ? column(a.col_exponents[c]) : 1.f) * inv);
}

// The first CTAs take the parts of the table, the next a.n scale a row of activations
// each, the others take eight rows of W.
template <int XT>
__global__ void __launch_bounds__(kThreads) prepare_kernel(ScaleRows a, RowPowers p)
{
    pdl_release();
    const long long cta = (long long)blockIdx.x - (p.table_top ? kTableParts : 0);
    if (cta < 0) {
        table_part(p, blockIdx.x);
    } else if (cta < a.n) {
        scale_row<XT>(a, cta);
    } else {
        const long long r = (cta - a.n) * (kThreads / 32) + (threadIdx.x >> 5);
        if (r < p.rows) row_power(p, r);
    }
    // The grid ends after the launch that it ran beside: one CTA waits for that (if all
    // did, they would hold the places of the rows behind them).
    if (blockIdx.x == gridDim.x - 1) pdl_wait();
}

// One CTA per row (or several rows in turn); eight elements per thread and step, read
// one by one (the rows start anywhere), written together.
__global__ void __launch_bounds__(kThreads) copy16_kernel(const uint16_t* x, long long ldx, long long n, long long cols,
                                                          uint16_t* out, long long ldo)
{
    pdl_release();
    for (long long r = blockIdx.x; r < n; r += gridDim.x)
        for (long long c = 8ll * threadIdx.x; c < cols; c += 8 * kThreads) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < cols && TCQ_IN_BOUNDS(r * ldx + c + i, (n - 1) * ldx + cols) ? x[r * ldx + c + i] : 0u;
            if (TCQ_IN_BOUNDS(r * ldo + c + 7, n * ldo))
                *reinterpret_cast<uint4*>(out + r * ldo + c) =
                    make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
        }
    if (blockIdx.x == gridDim.x - 1) pdl_wait();  // as above
}

}  // namespace

cudaError_t launch_prepare(ScaleRows a, RowPowers p, cudaStream_t stream)
{
    a.vec = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.ldx % 8 == 0;
    const long long grid = (p.table_top ? kTableParts : 0) + a.n + (p.rows + kThreads / 32 - 1) / (kThreads / 32);
    return launch_pdl(a.xdtype == TCQ_X_BF16 ? prepare_kernel<TCQ_X_BF16> : prepare_kernel<TCQ_X_F16>,
                      dim3((unsigned)grid), dim3(kThreads), 0, stream, a.early, a, p);
}

cudaError_t launch_copy16(const void* x, long long ldx, long long n, long long cols, void* out, long long ldo,
                          int num_sms, cudaStream_t stream)
{
    const long long grid = n < 32ll * num_sms ? n : 32ll * num_sms;
    return launch_pdl(copy16_kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, true,
                      static_cast<const uint16_t*>(x), ldx, n, cols, static_cast<uint16_t*>(out), ldo);
}

}  // namespace tcq
