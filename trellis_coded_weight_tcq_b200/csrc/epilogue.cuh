// epilogue.cuh -- a product's epilogue on sums that come from memory (the pieces of a
// cut reduction), four columns per lane.
#pragma once

#include "gemm.cuh"
#include "powers.cuh"
#include "q8.cuh"

namespace tcq {

// Outputs (t, r .. r + 3) of [tokens, rows], those below `rows`, from their sums: the powers
// of two, bias, 8-bit checkpoint, activation and residual, rounded once.  All lanes of a warp have the
// same t and consecutive quads, eight lanes a group of 32.  `vec`: out and residual rows
// that 8-byte accesses can reach.
template <int XT>
__device__ __forceinline__ void finish_quad(const Epilogue& e, long long t, long long r, long long tokens, long long rows,
                                            float (&v)[4], bool vec)
{
    const int lane = threadIdx.x & 31;
    const int count = rows - r < 4 ? (rows - r > 0 ? (int)(rows - r) : 0) : 4;
    const int row_exponent = e.row_scale && TCQ_IN_BOUNDS(t, tokens) ? exponent_of(__ldcg(e.row_scale + t)) : 0;
    const TableParts parts(e.table_top);
    float column[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        column[i] = i < count && e.col_scale && TCQ_IN_BOUNDS(r + i, rows) ? __ldcg(e.col_scale + r + i) : 1.f;
        bias[i] = i < count && e.bias && TCQ_IN_BOUNDS(r + i, rows) ? __ldg(e.bias + r + i) : 0.f;
    }
    const float table = parts.power();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = power_halves(row_exponent + exponent_of(power_product(column[i], table)));
        v[i] = fmaf(v[i] * p.x, p.y, bias[i]);
    }
    if (e.z_codes) {  // a group of 32 is eight lanes
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool int8 = e.z_format == TCQ_Q8_INT8;
        const uint32_t byte = int8 ? q8_scale_byte<TCQ_Q8_INT8>(top) : q8_scale_byte<TCQ_Q8_E4M3>(top);
        const float inv = q8_inv(byte);
        if (count > 0 && (lane & 7) == 0 && TCQ_IN_BOUNDS(t * ((rows + 31) / 32) + r / 32, tokens * ((rows + 31) / 32))) e.z_scales[t * ((rows + 31) / 32) + r / 32] = (uint8_t)byte;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count && TCQ_IN_BOUNDS(t * rows + r + i, tokens * rows))
                e.z_codes[t * rows + r + i] = byte == 255u ? 0 : (uint8_t)(int8 ? q8_encode<TCQ_Q8_INT8>(v[i], inv)
                                                                              : q8_encode<TCQ_Q8_E4M3>(v[i], inv));
    }
    act_values(v, e.act);
    if (count > 0 && !(TCQ_IN_BOUNDS(t * e.ldo + r + count - 1, (tokens - 1) * e.ldo + rows) &&
                       (!e.residual || TCQ_IN_BOUNDS(t * e.ldr + r + count - 1, (tokens - 1) * e.ldr + rows))))
        return;
    uint16_t* out = static_cast<uint16_t*>(e.out) + t * e.ldo + r;
    const uint16_t* res = e.residual ? static_cast<const uint16_t*>(e.residual) + t * e.ldr + r : nullptr;
    if (vec && count == 4) {
        if (res) {
            const uint2 q = *reinterpret_cast<const uint2*>(res);
            const float2 a = x_unpack2<XT>(q.x), b = x_unpack2<XT>(q.y);
            v[0] += a.x; v[1] += a.y; v[2] += b.x; v[3] += b.y;
        }
        *reinterpret_cast<uint2*>(out) = make_uint2(x_pack2<XT>(v[0], v[1]), x_pack2<XT>(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) out[i] = x_bits<XT>(res ? v[i] + x_load<XT>(res, i) : v[i]);
    }
}

// The fp32 outputs of the weight gradient.
__device__ __forceinline__ void finish_quad_f32(const Epilogue& e, long long t, long long r, long long tokens,
                                                long long rows, const float (&v)[4])
{
    float* out = static_cast<float*>(e.out) + t * e.ldo + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r + i < rows && TCQ_IN_BOUNDS(t * e.ldo + r + i, (tokens - 1) * e.ldo + rows)) out[i] = e.accumulate ? out[i] + v[i] : v[i];
}

}  // namespace tcq
