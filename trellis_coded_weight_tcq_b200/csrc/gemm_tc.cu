// gemm_tc.cu -- the 16-bit matrix products of the batched layer on the
// fifth-generation tensor cores.
//
// One kernel serves the three products; they differ in which operands run along
// the reduction (the tensor core reads either order from 128-byte swizzled tiles)
// and in the epilogue.  A pair of CTAs (a cluster of two, cta_group::2) computes a
// 256 x 256 tile: each CTA loads its half of both operands by TMA, 128 x 64 elements
// of each per stage, six stages deep (192 KB), and one thread of the first CTA issues
// the pair's MMAs (256 x 256 x 16).  The accumulators take 256 columns of each CTA's
// tensor memory; two sets of them let the epilogue warps store a tile while the
// next one is multiplied.  The grid is persistent, one pair per two SMs.
//
// Outputs that TMA can address (16-byte aligned base and rows) leave through shared
// memory: a warp writes 32 rows of 128 bytes to a swizzled box and stores it as whole
// lines (a lane's own 16-byte stores would each touch half a sector of 32 different
// rows); other outputs leave the box row by row.
//
// The tensor core's running fp32 sum loses about 1e-7 of a sum per square root of its
// steps.  That does not show in 16-bit outputs; the weight gradient, fp32 and summed over
// all tokens, takes its sums out of tensor memory every 1280 tokens at most and adds them
// in registers (root mean square error against float64 at 4096 tokens, relative to the
// gradient's: 1.6e-6 without, 2.9e-7 with; 8e-7 for 1111 tokens, one such sum).
//
// Measured on a B200, 4096 tokens through 14336 x 4096 (481 GFLOP), each launch by itself,
// with the second kernel: forward with GELU 323 us, input gradient 318 us, weight gradient
// 338 us (83, 86 and 75 % of the tensor pipe); the vendor library's bare products take 324 to
// 360 us there.  In runs of a second the board's power limit holds the SM clock at 1.4 to
// 1.5 GHz of 1.965 and whole calls take 413 to 420 us (weight gradient 395), so what costs energy
// costs time: the order of the tiles took 50 us off the weight gradient, whose kernel spills
// 12 bytes beside its 128 running sums.  Clock stamps: a
// stage takes 571 cycles of the pipe's 512 in the input gradient; the gap is the latency of
// loads behind a ring of six (a seventh stage does not fit beside the boxes).
//
// The last round of tiles, where it has work for half the pairs or fewer: a reduction is cut
// into as many pieces as there are pairs for, each writes its fp32 sums to the workspace,
// and a second kernel adds a tile's pieces in order and applies the epilogue (32 tokens
// through the input gradient of a 14336 x 4096 matrix have 16 tiles of 224 stages: four
// pieces; 4096 tokens have 256, three rounds of 74 and 34 more: two pieces each).
//
// Roles: warp 0 TMA, warp 1 MMA (first CTA of the pair only), warp 2 tensor memory,
// warps 4 and up epilogue.  Barriers: full (both CTAs' loads of a stage landed; in the
// first CTA), empty (the MMAs that read a stage are done; in both, by a commit to
// both), tfull / tempty (an accumulator set is complete / has been read).
#include "epilogue.cuh"
#include "gemm.cuh"
#include "pdl.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace tcq {

namespace {

// A tensor map of a row-major matrix, elements of 2 or 4 bytes.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, int element, const void* base, long long rows, long long cols,
              long long ld, int box_cols, int box_rows, CUtensorMapSwizzle swizzle)
{
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * element};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t step[2] = {1u, 1u};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map_out(CUtensorMap* map, const void* base, long long rows, long long cols, long long ld, int element)
{
    return make_map(map, element == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, element, base,
                    rows, cols, ld, 128 / element, 32, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool make_map_16bit(CUtensorMap* map, const void* base, long long rows, long long cols, long long ld, int box_rows)
{
    // the element type only matters for the fill, which is zero in both
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, rows, cols, ld, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool make_map_words(CUtensorMap* map, const void* base, long long rows, long long cols, int box_cols, int box_rows)
{
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, base, rows, cols, cols, box_cols, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
}

namespace {

constexpr int kStages = 6;
constexpr int kTile = 256;            // rows and columns of a pair's tile
constexpr int kDepth = 64;            // reduction depth of a stage
constexpr int kHalfBytes = 128 * kDepth * 2;  // one CTA's half of one operand's stage
constexpr int kBoxBytes = 32 * 128;   // a warp's box of the output: 32 rows of 128 bytes
constexpr int kSegment = 20;          // stages (1280 deep) at most that the weight gradient sums in tensor memory

// The input gradient has four epilogue warps with two boxes each.  The others have eight
// with one box, a half of the tile's columns each: the weight gradient's hold their sums in
// registers, and four would take longer over the forward product's activations than the
// tensor cores over the next tile (41k cycles against 37k for 4096 deep tiles, GELU).
__host__ __device__ constexpr int epilogue_warps(int kind) { return kind == kGemmDgrad ? 4 : 8; }
__host__ __device__ constexpr int gemm_threads(int kind) { return 128 + 32 * epilogue_warps(kind); }

struct __align__(1024) Smem {
    unsigned char a[kStages][kHalfBytes];
    unsigned char b[kStages][kHalfBytes];
    unsigned char box[8][kBoxBytes];
    float4 cols[kTile / 2];  // the powers of two and the biases of two columns of a tile
    unsigned long long full[kStages], empty[kStages], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int stop;
};

static_assert(sizeof(Smem) <= 227 * 1024, "shared memory");

struct Shape {
    long long m, n, k;
    int m_tiles, n_tiles, k_steps;
    int fmt;
    int whole;   // tiles that are summed whole; the others' reductions are cut into
    int pieces;  // pieces, whose sums go to the workspace
    int across;  // neighbouring tiles of the order that run along one axis (tile_at)
    bool rows_first;  // that axis is the rows'
};

// A pair's next piece of work: its tile's first row and column, its stages, and its place
// in the workspace (-1: the whole tile).
struct Item {
    int m0, n0, k0, k1, slot;
};

// First row and column of a tile.  The order goes through bands of `across` tiles along
// one axis, all of the other axis in each band, so that the tiles that run at a time share
// their operands in L2 (tile_order).
__device__ __forceinline__ int2 tile_at(const Shape& p, int tile)
{
    const int u_tiles = p.rows_first ? p.m_tiles : p.n_tiles, v_tiles = p.rows_first ? p.n_tiles : p.m_tiles;
    const int band = tile / (p.across * v_tiles), in_band = tile - band * p.across * v_tiles;
    const int left = u_tiles - band * p.across, width = left < p.across ? left : p.across;
    const int v = in_band / width, u = band * p.across + in_band - v * width;
    return p.rows_first ? make_int2(u * kTile, v * kTile) : make_int2(v * kTile, u * kTile);
}

__device__ __forceinline__ Item work_item(const Shape& p, int t)
{
    const int slot = t - p.whole;
    const int tile = slot < 0 ? t : p.whole + slot / p.pieces, piece = slot < 0 ? 0 : slot % p.pieces;
    const int2 at = tile_at(p, tile);
    if (slot < 0) return {at.x, at.y, 0, p.k_steps, -1};
    return {at.x, at.y, (int)((long long)p.k_steps * piece / p.pieces), (int)((long long)p.k_steps * (piece + 1) / p.pieces),
            slot};
}

// Stages between two accumulator sets: all, or in the weight gradient equal parts of at
// most kSegment.
template <int KIND>
__device__ __forceinline__ int segment_of(const Item& w)
{
    const int n = w.k1 - w.k0;
    if (KIND != kGemmWgrad || n <= kSegment) return n;
    const int parts = (n + kSegment - 1) / kSegment;
    return (n + parts - 1) / parts;
}

// 32 values of one row through the epilogue: row r of m, columns c .. c + 31, `count` of them
// below n.
template <int KIND, int XT>
__device__ __forceinline__ void apply32(const Epilogue& e, long long r, long long c, long long m, long long n, float (&v)[32],
                                        int count, int row_exponent, const float4* cols,
                                        const unsigned char* box_row, int half)
{
    if constexpr (KIND == kGemmDgrad) {
        if (e.row_scale || e.table_top) {
            const float2 h = power_halves(row_exponent);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
                f2_split(f2_mul(f2_mul(f2(v[i], v[i + 1]), f2(h.x, h.x)), f2(h.y, h.y)), v[i], v[i + 1]);
        }
    }
    if constexpr (KIND == kGemmForward) {
        if (e.row_scale) {  // the row's and the column's powers together: each alone may pass fp32's range
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float4 p = cols[i / 2];
                const float2 a = power_halves(row_exponent + exponent_of(p.x)), b = power_halves(row_exponent + exponent_of(p.y));
                v[i] = fmaf(v[i] * a.x, a.y, p.z);
                v[i + 1] = fmaf(v[i + 1] * b.x, b.y, p.w);
            }
        } else if (e.col_scale || e.table_top || e.bias) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {  // two columns per 16-byte read, the same in every lane
                const float4 p = cols[i / 2];
                f2_split(f2_fma(f2(v[i], v[i + 1]), f2(p.x, p.y), f2(p.z, p.w)), v[i], v[i + 1]);
            }
        }
        if (e.z_codes) {
            const long long group = r * ((n + 31) / 32) + c / 32;
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < count) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
            uint8_t* z = e.z_codes + r * n + c;
            const bool int8 = e.z_format == TCQ_Q8_INT8;
            const uint32_t byte = int8 ? q8_scale_byte<TCQ_Q8_INT8>(top) : q8_scale_byte<TCQ_Q8_E4M3>(top);
            const float inv = q8_inv(byte);
            if (TCQ_IN_BOUNDS(group, m * ((n + 31) / 32))) e.z_scales[group] = (uint8_t)byte;
            uint32_t code[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) code[i] = 0u;
            if (byte != 255u) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t q = int8 ? q8_encode<TCQ_Q8_INT8>(v[i], inv) : q8_encode<TCQ_Q8_E4M3>(v[i], inv);
                    code[i / 4] |= q << (8 * (i & 3));
                }
            }
            const bool in = TCQ_IN_BOUNDS(r * n + c + count - 1, m * n);
            if (in && count == 32 && (reinterpret_cast<uintptr_t>(z) & 15) == 0) {
                reinterpret_cast<uint4*>(z)[0] = make_uint4(code[0], code[1], code[2], code[3]);
                reinterpret_cast<uint4*>(z)[1] = make_uint4(code[4], code[5], code[6], code[7]);
            } else if (in) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i < count) z[i] = (uint8_t)(code[i / 4] >> (8 * (i & 3)));
            }
        }
        act_values(v, e.act);
        if (e.residual) {  // from the warp's box (load_rows)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 t = *reinterpret_cast<const uint4*>(box_row + (((4 * half + i) ^ (threadIdx.x & 7)) << 4));
                const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float2 f = x_unpack2<XT>(w[h]);
                    v[8 * i + 2 * h] += f.x;
                    v[8 * i + 2 * h + 1] += f.y;
                }
            }
        }
    }
}

// A box's rows to outputs that TMA cannot address, row by row: neighbouring lanes store
// neighbouring elements (2 or 4 bytes each).  The box starts `at` elements into `base`,
// which has `most`.
template <typename T>
__device__ __forceinline__ void store_rows(const unsigned char* box, T* base, long long at, long long most, long long ldo,
                                           int rows, int cols, int lane)
{
    T* out = base + at;
    constexpr int per = 128 / sizeof(T), ahead = 8 * 32 / per;  // columns of a box, rows read together
#pragma unroll 1
    for (int i0 = 0; i0 < rows; i0 += ahead) {
        T v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * 32 / per, byte = (lane + j * 32 % per) * (int)sizeof(T);
            v[j] = *reinterpret_cast<const T*>(box + i * 128 + ((((byte >> 4) ^ (i & 7)) << 4) | (byte & 15)));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * 32 / per, c = lane + j * 32 % per;
            if (i < rows && c < cols && TCQ_IN_BOUNDS(at + i * ldo + c, most)) out[i * ldo + c] = v[j];
        }
    }
}

// The reverse: a box from 16-bit rows.  `vec`: rows of whole 16-byte vectors, eight lanes a
// row, all loads in flight together (a lane's own row would take 32 sectors per load).
__device__ __forceinline__ void load_rows(unsigned char* box, const uint16_t* base, long long at, long long most, long long ld,
                                          int rows, int cols, int lane, bool vec)
{
    const uint16_t* in = base + at;
    if (vec) {
        const int c = lane & 7;
        uint4 t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            t[i] = r < rows && 8 * c < cols && TCQ_IN_BOUNDS(at + r * ld + 8 * c + 7, most) ? *reinterpret_cast<const uint4*>(in + r * ld + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            *reinterpret_cast<uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4)) = t[i];
        }
        return;
    }
#pragma unroll 4
    for (int i = 0; i < rows; ++i) {
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
            const int c = lane + h, byte = 2 * c;
            *reinterpret_cast<uint16_t*>(box + i * 128 + ((((byte >> 4) ^ (i & 7)) << 4) | (byte & 15))) =
                c < cols && TCQ_IN_BOUNDS(at + i * ld + c, most) ? in[i * ld + c] : (uint16_t)0;
        }
    }
}

// 64 bytes of a lane's row of a swizzled box: 32 16-bit values, the first or second half.
template <int XT>
__device__ __forceinline__ void box32(unsigned char* row, int lane, int half, const float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(row + (((4 * half + i) ^ (lane & 7)) << 4)) =
            make_uint4(x_pack2<XT>(v[8 * i], v[8 * i + 1]), x_pack2<XT>(v[8 * i + 2], v[8 * i + 3]),
                       x_pack2<XT>(v[8 * i + 4], v[8 * i + 5]), x_pack2<XT>(v[8 * i + 6], v[8 * i + 7]));
}

template <int KIND, int XT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(gemm_threads(KIND), 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_sums, Shape p, Epilogue e,
            bool vec, bool tma_out, unsigned int* err)
{
    // map_sums: the workspace, [slot, 256 rows] x 256 columns, fp32
    constexpr int AMN = KIND == kGemmWgrad, BMN = KIND != kGemmForward, EW = epilogue_warps(KIND);
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem& S = *reinterpret_cast<Smem*>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int items = p.whole + (p.m_tiles * p.n_tiles - p.whole) * p.pieces;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&S.full[i]), 1);
            mbar_init(smem_addr(&S.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&S.tfull[i]), 1);
            mbar_init(smem_addr(&S.tempty[i]), 2 * EW);  // the epilogue warps of both CTAs
        }
        mbar_init(smem_addr(&S.drain), 1);
        S.stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
    }
    if (warp == 2) tmem_alloc<2>(smem_addr(&S.tmem), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    pdl_wait();  // the operands, and the workspace that the call before may have used
    pdl_release();
    const uint32_t tmem = S.tmem;
    volatile int* stop = &S.stop;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = pair; t < items && ok; t += pairs) {
                const Item w = work_item(p, t);
                const int m0 = w.m0 + (int)rank * 128, n0 = w.n0 + (int)rank * 128;
                for (int ks = w.k0; ks < w.k1; ++ks, ++it) {
                    const int s = it % kStages;
                    ok = mbar_wait(smem_addr(&S.empty[s]), ((it / kStages) & 1) ^ 1, stop, err);
                    if (!ok) break;
                    const uint32_t full = map_to_cta(smem_addr(&S.full[s]), 0);
                    if (rank == 0) mbar_expect_tx(smem_addr(&S.full[s]), 4 * kHalfBytes);
                    const int k0 = ks * kDepth;
                    const uint32_t a = smem_addr(S.a[s]), b = smem_addr(S.b[s]);
                    if constexpr (AMN) {
                        tma_load_2d_pair(a, &map_a, full, m0, k0);
                        tma_load_2d_pair(a + kHalfBytes / 2, &map_a, full, m0 + 64, k0);
                    } else {
                        tma_load_2d_pair(a, &map_a, full, k0, m0);
                    }
                    if constexpr (BMN) {
                        tma_load_2d_pair(b, &map_b, full, n0, k0);
                        tma_load_2d_pair(b + kHalfBytes / 2, &map_b, full, n0 + 64, k0);
                    } else {
                        tma_load_2d_pair(b, &map_b, full, k0, n0);
                    }
                }
            }
            // after a stop, what was loaded last is still waited for
            if (*stop && rank == 0)
                for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
                    mbar_drain(smem_addr(&S.full[i % kStages]), (i / kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        if (lane == 0) {
            const uint32_t idesc = mma_idesc(256, 256, p.fmt, AMN, BMN);
            int it = 0, done = 0;
            bool ok = true;
            for (int t = pair; t < items && ok; t += pairs) {
                const Item w = work_item(p, t);
                const int segment = segment_of<KIND>(w);
                for (int k0 = w.k0; k0 < w.k1 && ok; k0 += segment, ++done) {
                    const int acc = done & 1;
                    ok = mbar_wait(smem_addr(&S.tempty[acc]), ((done >> 1) & 1) ^ 1, stop, err);
                    if (!ok) break;
                    tc_fence_after();
                    const int k1 = w.k1 - k0 > segment ? k0 + segment : w.k1;
                    for (int ks = k0; ks < k1; ++ks, ++it) {
                        const int s = it % kStages;
                        ok = mbar_wait(smem_addr(&S.full[s]), (it / kStages) & 1, stop, err);
                        if (!ok) break;
                        tc_fence_after();
                        // 16 deep: 32 bytes along a K-major row, 16 rows of 128 bytes otherwise
                        // (a descriptor counts in 16 bytes)
                        const unsigned long long da = smem_desc_sw128(smem_addr(S.a[s]), kHalfBytes / 2);
                        const unsigned long long db = smem_desc_sw128(smem_addr(S.b[s]), kHalfBytes / 2);
#pragma unroll
                        for (int j = 0; j < kDepth / 16; ++j)
                            mma_f16<2>(tmem + acc * 256, da + j * (AMN ? 128 : 2), db + j * (BMN ? 128 : 2), idesc,
                                       ks != k0 || j != 0);
                        mma_commit<2>(smem_addr(&S.empty[s]));
                    }
                    if (ok) mma_commit<2>(smem_addr(&S.tfull[acc]));
                }
            }
            if (*stop) {  // nothing issued may still run when the tensor memory is freed
                mma_commit<2>(smem_addr(&S.drain));
                mbar_drain(smem_addr(&S.drain), 0);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const float table = KIND != kGemmWgrad ? table_power(e.table_top) : 1.f;
        int done = 0;
        unsigned turn = 0;  // of the warp's boxes: the next one's last store is then the oldest
        bool ok = true;
        for (int t = pair; t < items && ok; t += pairs) {
            const Item w = work_item(p, t);
            // rows and columns in the output, or in the workspace
            const bool cut = w.slot >= 0;
            const int out_row = cut ? w.slot * kTile : w.m0, out_col = cut ? 0 : w.n0;
            if constexpr (KIND == kGemmWgrad) {
                const int half = (warp - 4) >> 2;
                unsigned char* box = S.box[warp - 4];
                float sum[128];
#pragma unroll
                for (int i = 0; i < 128; ++i) sum[i] = 0.f;
                const int segment = segment_of<KIND>(w);
                for (int k0 = w.k0; k0 < w.k1 && ok; k0 += segment, ++done) {
                    const int acc = done & 1;
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&S.tfull[acc]), (done >> 1) & 1, stop, err));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {  // eight at a time: registers are full
                        float v[8];
                        tmem_load8(lanes + acc * 256 + 128 * half + 8 * j, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum[8 * j + i] += v[i];
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_addr(&S.tempty[acc]), 0));
                }
                if (!ok) break;
                const int local = (int)rank * 128 + quarter * 32, r0 = w.m0 + local;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = w.n0 + 128 * half + 32 * j;
                    if (c >= p.n || r0 >= p.m) break;  // the same in every lane
                    const bool plain = !tma_out && !cut;
                    if (plain && e.accumulate && r0 + lane < p.m) {
                        const float* o = static_cast<const float*>(e.out) + (long long)(r0 + lane) * e.ldo + c;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < p.n && TCQ_IN_BOUNDS((long long)(r0 + lane) * e.ldo + c + i, (p.m - 1) * e.ldo + p.n))
                                sum[32 * j + i] += o[i];
                    }
                    {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4*>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                                make_float4(sum[32 * j + 4 * i], sum[32 * j + 4 * i + 1], sum[32 * j + 4 * i + 2],
                                            sum[32 * j + 4 * i + 3]);
                        if (!plain) fence_async_shared();
                        __syncwarp();
                        if (plain) {
                            store_rows(box, static_cast<float*>(e.out), (long long)r0 * e.ldo + c, (p.m - 1) * e.ldo + p.n,
                                       e.ldo, p.m - r0 < 32 ? (int)(p.m - r0) : 32, p.n - c < 32 ? (int)(p.n - c) : 32, lane);
                            __syncwarp();
                        } else if (lane == 0) {
                            if (e.accumulate && !cut)
                                tma_add_2d(&map_out, smem_addr(box), c, r0);
                            else
                                tma_store_2d(cut ? &map_sums : &map_out, smem_addr(box), out_col + c - w.n0, out_row + local);
                            bulk_commit();
                        }
                    }
                }
            } else {
                constexpr int boxes = 8 / EW, span = kTile * 4 / EW;  // a warp's boxes and columns
                const int c0 = (warp - 4) / 4 * span;
                const int local = (int)rank * 128 + quarter * 32;
                const long long r0 = w.m0 + local, r = r0 + lane, n0 = w.n0;
                const int acc = done & 1;
                if constexpr (KIND == kGemmForward) {
                    // this tile's columns, while its product still runs
                    named_barrier(1, 32 * EW);  // the last tile's have been read
                    for (int i = threadIdx.x - 128; i < kTile; i += 32 * EW) {
                        const long long c = n0 + i;
                        float* at = reinterpret_cast<float*>(S.cols + i / 2) + (i & 1);
                        at[0] = power_product(e.col_scale && c < p.n ? __ldcg(e.col_scale + c) : 1.f, table);
                        at[2] = e.bias && c < p.n ? __ldg(e.bias + c) : 0.f;
                    }
                }
                // a box of the residual: each half's values make room for that half's outputs
                const int rows = p.m - r0 < 32 ? (int)(p.m - r0) : 32;
                auto residual_box = [&](unsigned char* box, int c) {
                    if (lane == 0) bulk_wait_read<boxes - 1>();
                    __syncwarp();
                    load_rows(box, static_cast<const uint16_t*>(e.residual), r0 * e.ldr + n0 + c,
                              (p.m - 1) * e.ldr + p.n, e.ldr, rows,
                              p.n - n0 - c < 64 ? (int)(p.n - n0 - c) : 64, lane, vec);
                    __syncwarp();
                };
                const bool residual = KIND == kGemmForward && e.residual && !cut;
                if (residual && r0 < p.m && n0 + c0 < p.n) residual_box(S.box[(warp - 4) * boxes + (turn & (boxes - 1))], c0);
                ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&S.tfull[acc]), (done >> 1) & 1, stop, err));
                // the columns are there; after a wait that gave up all warps stop together, or
                // the others would wait at the next barrier
                if constexpr (KIND == kGemmForward) ok = named_all(1, 32 * EW, ok);
                if (!ok) break;
                tc_fence_after();
                const int row_exponent = (e.row_scale && r < p.m ? exponent_of(__ldcg(e.row_scale + r)) : 0) +
                                         (KIND == kGemmDgrad ? exponent_of(table) : 0);
                if (cut) {  // the sums as they are, 32 columns at a time
#pragma unroll 1
                    for (int c = c0; c < c0 + span; c += 32) {
                        if (n0 + c >= p.n || r0 >= p.m) break;
                        unsigned char* box = S.box[(warp - 4) * boxes + (turn++ & (boxes - 1))];
                        float v[32];
                        tmem_load32(lanes + acc * 256 + c, v);
                        if (lane == 0) bulk_wait_read<boxes - 1>();
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4*>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&map_sums, smem_addr(box), c, out_row + local);
                            bulk_commit();
                        }
                    }
                }
#pragma unroll 1
                for (int c = cut ? c0 + span : c0; c < c0 + span; c += 64) {
                    if (n0 + c >= p.n || r0 >= p.m) break;  // the same in every lane
                    unsigned char* box = S.box[(warp - 4) * boxes + (turn++ & (boxes - 1))];
                    const int cols = p.n - n0 - c < 64 ? (int)(p.n - n0 - c) : 64;
                    if (residual && c != c0) residual_box(box, c);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const long long ch = n0 + c + 32 * h;
                        if (ch >= p.n) break;
                        float v[32];
                        tmem_load32(lanes + acc * 256 + c + 32 * h, v);
                        const int count = p.n - ch < 32 ? (int)(p.n - ch) : 32;
                        if (r < p.m) apply32<KIND, XT>(e, r, ch, p.m, p.n, v, count, row_exponent,
                                                       S.cols + (c + 32 * h) / 2, box + lane * 128, h);
                        if (h == 0 && !residual) {  // the box's last store has been read
                            if (lane == 0) bulk_wait_read<boxes - 1>();
                            __syncwarp();
                        }
                        box32<XT>(box + lane * 128, lane, h, v);
                        __syncwarp();
                    }
                    if (tma_out) {
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&map_out, smem_addr(box), (int)(n0 + c), (int)r0);
                            bulk_commit();
                        }
                    } else {
                        store_rows(box, static_cast<uint16_t*>(e.out), r0 * e.ldo + n0 + c, (p.m - 1) * e.ldo + p.n, e.ldo,
                                   rows, cols, lane);
                        __syncwarp();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_cta(smem_addr(&S.tempty[acc]), 0));
                ++done;
            }
        }
        if (lane == 0) bulk_wait_all();  // the boxes are read and the outputs written
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        tmem_free<2>(tmem, 512);
    }
}

// Adds a tile's pieces in order and applies the epilogue: a warp takes 128 columns of a row.
template <int KIND, int XT>
__global__ void __launch_bounds__(256) finish_kernel(Shape p, Epilogue e, const float* partial, bool vec)
{
    const int lane = threadIdx.x & 31, tile = p.whole + blockIdx.x;
    const int local = blockIdx.y * 8 + (threadIdx.x >> 5), c = blockIdx.z * 128 + 4 * lane;
    const int2 at = tile_at(p, tile);
    const long long r = (long long)at.x + local, n0 = at.y;
    pdl_wait();
    if (r >= p.m || n0 + blockIdx.z * 128 >= p.n) return;
    const float* src = partial + ((long long)blockIdx.x * p.pieces * kTile + local) * kTile + c;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < p.pieces; ++i) {
        if (!TCQ_IN_BOUNDS(src - partial + (long long)i * kTile * kTile + 3,
                           ((long long)p.m_tiles * p.n_tiles - p.whole) * p.pieces * kTile * kTile))
            break;
        const float4 d = __ldcg(reinterpret_cast<const float4*>(src + (long long)i * kTile * kTile));
        v[0] += d.x; v[1] += d.y; v[2] += d.z; v[3] += d.w;
    }
    if constexpr (KIND == kGemmWgrad)
        finish_quad_f32(e, r, n0 + c, p.m, p.n, v);
    else
        finish_quad<XT>(e, r, n0 + c, p.m, p.n, v, vec);
}

// The order of the tiles.  The axis with fewer tiles goes first: where its operand is
// small enough to stay in L2 the other is read once (DRAM reads of the weight gradient of
// 4096 tokens, 14336 x 4096: 1440 MB the other way round, 235 MB and 400 -> 347 us so).  Where it is not,
// bands of about the square root of the tiles that run at a time read the least.
void tile_order(Shape& s, int pairs)
{
    constexpr long long kStays = 48ll << 20;
    s.rows_first = s.m_tiles <= s.n_tiles;
    const int tiles = s.rows_first ? s.m_tiles : s.n_tiles;
    int root = 1;
    while ((root + 1) * (root + 1) <= pairs) ++root;
    s.across = 2ll * kTile * s.k * tiles <= kStays || tiles < root ? tiles : root;
}

// The tiles that whole rounds of the pairs leave over are cut where that saves more than
// it costs, into the pieces that save the most.  A cut into p pieces saves k - k / p stages
// (0.3 us each); writing and adding the sums costs as much as 5 stages and 2/9 of one per
// piece (measured with 2 to 72 pieces, within 0.5 us).  Whole / cut, in us: 4 tiles, 16
// stages 14.0 / 12.3; 32 tiles, 32 stages 21.8 / 22.6, 64 stages 33.6 / 30.0; 88 tiles (14
// left) 24 stages 26.5 / 28.1, 64 stages 53.5 / 44.1.
void cut_rest(Shape& s, int pairs)
{
    const long long tiles = (long long)s.m_tiles * s.n_tiles;
    const int rest = (int)(tiles % pairs), k = s.k_steps;
    s.whole = (int)tiles;
    s.pieces = 1;
    if (rest == 0) return;
    long long best = 0;
    for (int p = 2; p <= pairs / rest && p <= k; ++p) {
        const long long gain = 9ll * (k - (k + p - 1) / p) - 45 - 2 * rest * p;
        if (gain > best) {
            best = gain;
            s.whole = (int)(tiles - rest);
            s.pieces = p;
        }
    }
}

Shape shape_of(long long m, long long n, long long k, int num_sms)
{
    Shape s = {};
    s.m = m;
    s.n = n;
    s.k = k;
    s.m_tiles = (int)((m + kTile - 1) / kTile);
    s.n_tiles = (int)((n + kTile - 1) / kTile);
    s.k_steps = (int)((k + kDepth - 1) / kDepth);
    tile_order(s, num_sms / 2);
    cut_rest(s, num_sms / 2);
    return s;
}

long long slots(const Shape& s) { return s.pieces > 1 ? ((long long)s.m_tiles * s.n_tiles - s.whole) * s.pieces : 0; }

template <int KIND, int XT>
cudaError_t launch(const GemmProblem& g, const Epilogue& e, float* partial, int num_sms, unsigned int* err,
                   cudaStream_t stream)
{
    const long long tiles = (g.m + kTile - 1) / kTile * ((g.n + kTile - 1) / kTile);
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    CUtensorMap ma, mb, mo, ms;
    const bool ok = (KIND == kGemmWgrad ? make_map_16bit(&ma, g.a, g.k, g.m, g.lda, 64)
                                        : make_map_16bit(&ma, g.a, g.m, g.k, g.lda, 128)) &&
                    (KIND == kGemmForward ? make_map_16bit(&mb, g.b, g.n, g.k, g.ldb, 128)
                                          : make_map_16bit(&mb, g.b, g.k, g.n, g.ldb, 64));
    if (!ok) return cudaErrorInvalidValue;
    Shape s = shape_of(g.m, g.n, g.k, num_sms);
    s.fmt = g.fmt;
    const int es = KIND == kGemmWgrad ? 4 : 2;
    bool vec = (reinterpret_cast<uintptr_t>(e.out) & 15) == 0 && e.ldo * es % 16 == 0;
    const bool tma_out = vec;
    mo = ms = ma;  // where they are not used
    if (tma_out && !make_map_out(&mo, e.out, g.m, g.n, e.ldo, es)) return cudaErrorInvalidValue;
    if (s.pieces > 1 && !make_map_out(&ms, partial, slots(s) * kTile, kTile, kTile, 4)) return cudaErrorInvalidValue;
    // the residual by 16-byte loads: rows of whole vectors
    if (e.residual)
        vec = (reinterpret_cast<uintptr_t>(e.residual) & 15) == 0 && e.ldr % 8 == 0 && g.n % 8 == 0;
    cudaError_t st = cudaFuncSetAttribute(gemm_kernel<KIND, XT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)sizeof(Smem));
    if (st != cudaSuccess) return st;
    const long long items = s.whole + (s.pieces > 1 ? slots(s) : 0);
    const int pairs = (int)(items < num_sms / 2 ? items : num_sms / 2);
    // every product comes after a launch of its own call (the decode, the unpacking)
    st = launch_pdl(gemm_kernel<KIND, XT>, dim3(2 * pairs), dim3(gemm_threads(KIND)), sizeof(Smem), stream, true, ma, mb, mo,
                    ms, s, e, vec, tma_out, err);
    if (st != cudaSuccess || s.pieces == 1) return st;
    // quads: 8-byte accesses
    bool quads = (reinterpret_cast<uintptr_t>(e.out) & 7) == 0 && e.ldo % 4 == 0;
    if (e.residual) quads = quads && (reinterpret_cast<uintptr_t>(e.residual) & 7) == 0 && e.ldr % 4 == 0;
    return launch_pdl(finish_kernel<KIND, XT>, dim3((unsigned)(tiles - s.whole), kTile / 8, kTile / 128), dim3(256), 0, stream, true, s,
                      e, static_cast<const float*>(partial), quads);
}

}  // namespace

size_t gemm_partial_bytes(long long m, long long n, long long k, int num_sms)
{
    if ((m + kTile - 1) / kTile * ((n + kTile - 1) / kTile) > INT32_MAX / 2) return 0;  // refused by the launch
    return (size_t)slots(shape_of(m, n, k, num_sms)) * kTile * kTile * sizeof(float);
}

cudaError_t launch_gemm_tc(GemmKind kind, const GemmProblem& p, const Epilogue& e, float* partial, int num_sms,
                           unsigned int* err, cudaStream_t stream)
{
    const bool bf = p.xdtype == TCQ_X_BF16;
    switch (kind) {
    case kGemmForward:
        return bf ? launch<kGemmForward, TCQ_X_BF16>(p, e, partial, num_sms, err, stream)
                  : launch<kGemmForward, TCQ_X_F16>(p, e, partial, num_sms, err, stream);
    case kGemmDgrad:
        return bf ? launch<kGemmDgrad, TCQ_X_BF16>(p, e, partial, num_sms, err, stream)
                  : launch<kGemmDgrad, TCQ_X_F16>(p, e, partial, num_sms, err, stream);
    default: return launch<kGemmWgrad, TCQ_X_F16>(p, e, partial, num_sms, err, stream);
    }
}

}  // namespace tcq
