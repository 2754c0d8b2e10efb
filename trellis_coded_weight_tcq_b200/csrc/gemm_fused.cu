// gemm_fused.cu -- the forward product for small batches: the matrix is decoded
// inside the product and never written out.
//
// With few tokens the product is bound by decoding (one shared-memory lookup per
// weight, about 3.5 bank passes per 32 random entries), so every weight is decoded
// once per 256 tokens and goes straight into a tensor-core operand tile.  The
// weights take the M side of the MMA: a CTA multiplies 128 rows of W by up to 256
// tokens, D[row, token] in tensor memory (cta_group::1, 128 x N x 16).
//
// 16 warps decode, in two groups that take turns at units of 128 columns (two stages
// of the ring): a warp covers 16 rows, lanes 0-15 the first stage's 64 columns of
// them, lanes 16-31 the second's.  A lane turns its 2 k stream words into eight 16-byte
// pieces of the swizzled K-major tile, held in registers until the stage is free.
// The look-ups leave the load/store pipe little room (46k of 88k cycles for 14336 x
// 4096, 71k with everything else), so the stream words come by TMA where shared memory
// and their alignment allow: boxes of 128 rows by a unit's words and the four before
// them, through a ring of their own; a warp's reads of 16 separate rows from global
// memory would take 16 passes each.  Otherwise a warp reads whole 32-byte sectors of its
// rows.  Warp 16 loads the activations' tiles, warp 18 the stream words, one thread of
// warp 17 issues the MMAs.
//
// Work is split over the SMs evenly, in units: a CTA takes a contiguous run of (tile,
// unit) pairs, so a tile's reduction may be cut into pieces; each writes its fp32 sums
// to the workspace, and a second kernel adds a tile's pieces in order and applies the
// epilogue.  The split depends on the shape and the SM count only.
#include "decode16.cuh"
#include "gemm.cuh"
#include "pdl.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace tcq {

namespace {

constexpr int kDecodeWarps = 16;
constexpr int kThreads = (kDecodeWarps + 3) * 32;
constexpr int kRows = 128;             // rows of W per tile
constexpr int kDepth = 64;             // columns per stage
constexpr int kABytes = kRows * kDepth * 2;
constexpr int kMaxSlots = 8;
constexpr int kMaxBoxes = 4;
constexpr int kSmemBytes = 227 * 1024;

struct Barriers {
    unsigned long long full[kMaxSlots], empty[kMaxSlots], tfull[2], tempty[2], drain;
    unsigned long long words_full[kMaxBoxes], words_empty[kMaxBoxes];
    uint32_t tmem;
    int stop;
    int fills[kMaxSlots];  // warps that have filled a slot, counted from the start
};

struct Plan {
    long long n;          // tokens
    int np;               // tokens per tile, a multiple of 16
    int row_tiles, token_tiles;
    int steps;            // units of 128 columns of a whole reduction
    long long units;      // tiles * steps
    int ctas;
    int pieces;           // slots per tile in the workspace
    int slots;            // ring depth
    int per;              // stages per slot: 2 (a unit), or 1 where only two stages fit
    int tmem_columns;
    int table;            // shared-memory bytes of the table, a multiple of 1024
    int boxes;            // depth of the stream words' ring, or 0: read from global memory
};

// the CTA that has unit u, and the first unit of a CTA
__host__ __device__ inline long long first_unit(const Plan& p, long long cta) { return p.units * cta / p.ctas; }
__host__ __device__ inline int cta_of(const Plan& p, long long u) { return (int)(((u + 1) * p.ctas - 1) / p.units); }

// 2 K stream words of a lane's 64 columns, in the widest loads their alignment allows
// (`wide`: the stream starts on a 16-byte boundary)
template <int K>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[2 * K], bool wide)
{
    if (!wide) {
#pragma unroll
        for (int i = 0; i < 2 * K; ++i) w[i] = __ldg(p + i);
    } else if constexpr (K % 2 == 0) {
#pragma unroll
        for (int i = 0; i < 2 * K; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + i));
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2 * K; i += 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + i));
            w[i] = v.x; w[i + 1] = v.y;
        }
    }
}

// Bytes of a row in a box of stream words: a unit's 4 k words and the four before them.
__host__ __device__ constexpr int box_row_bytes(int k) { return 16 * (k + 1); }

template <int K, int CODE>
__global__ void __launch_bounds__(kThreads, 1)
fused_kernel(CodedMatrix w, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_words,
             Plan p, const float* row_pow2, float* partial, unsigned int* err)
{
    constexpr int RB = box_row_bytes(K);
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* ring = sm + p.table;
    const int bbytes = p.np * kDepth * 2;
    const int sbytes = p.per * (kABytes + bbytes);  // a slot: its A stages, then its B stages
    unsigned char* boxes = ring + (size_t)p.slots * sbytes;
    Barriers& B = *reinterpret_cast<Barriers*>(boxes + p.boxes * kRows * RB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.slots; ++i) {
            mbar_init(smem_addr(&B.full[i]), kDecodeWarps / 2 + 1);  // a group's warps, and the TMA thread
            mbar_init(smem_addr(&B.empty[i]), 1);
            B.fills[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&B.tfull[i]), 1);
            mbar_init(smem_addr(&B.tempty[i]), kDecodeWarps);
        }
        for (int i = 0; i < p.boxes; ++i) {
            mbar_init(smem_addr(&B.words_full[i]), 1);
            mbar_init(smem_addr(&B.words_empty[i]), kDecodeWarps / 2);
        }
        mbar_init(smem_addr(&B.drain), 1);
        B.stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_x);
        if (p.boxes) tma_prefetch_map(&map_words);
    }
    if (warp == kDecodeWarps + 1) tmem_alloc<1>(smem_addr(&B.tmem), p.tmem_columns);
    stage_table<CODE>(sm, w.cb, w.cb_f16, w.L);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();  // the scaled activations and the row powers
    pdl_release();
    const uint32_t tmem = B.tmem;
    volatile int* stop = &B.stop;
    const long long u0 = first_unit(p, blockIdx.x), u1 = first_unit(p, blockIdx.x + 1);
    const int acc_columns = p.tmem_columns / 2;

    if (warp < kDecodeWarps) {
        const int group = warp >> 3, half = lane >> 4;
        const int r = (warp & 7) * 16 + (lane & 15);  // row of the tile
        const uint32_t mask = (1u << w.L) - 1u;
        const int T = w.T, cols = (int)w.cols, nb = cols / T;
        const int tshift = (T & (T - 1)) == 0 ? __ffs(T) - 1 : -1;
        const bool wide = (reinterpret_cast<uintptr_t>(w.bits) & 15) == 0;
        const int row_words = cols / 32 * K;
        // where the group's next unit is: its tile, its place in the reduction, its row
        long long tile = u0 / p.steps;
        int ks = (int)(u0 - tile * p.steps);
        const uint32_t* bits = nullptr;  // this lane's row, or none
        long long row = 0;
        float inv = 1.f;  // the row's power
        auto enter_tile = [&]() {
            row = (tile % p.row_tiles) * kRows + r;
            bits = row < w.rows ? w.bits + row * row_words : nullptr;
            if (bits && w.scale) inv = __ldg(row_pow2 + row);
        };
        auto advance = [&](int by) {
            for (ks += by; ks >= p.steps; ks -= p.steps) {
                ++tile;
                if (ks - p.steps < p.steps) enter_tile();
            }
        };
        enter_tile();
        advance(group);
        // The words of this lane's 64 columns, the word before them, their scale, the row's
        // inverse power, of the group's unit i (counted from u0).  Nothing here depends on
        // what was loaded from global memory, so that the loads stay in flight over the
        // decoding of the unit before.
        bool ok = true;
        auto fetch = [&](int i, uint32_t (&words)[2 * K], uint32_t& prev, float& sc, float& in) {
            const int c = ks * 128 + half * kDepth;
            const bool in_row = bits && c < cols;
            const int j = tshift >= 0 ? c >> tshift : c / T;
            const bool first = c == j * T;
            sc = 0.f;
            prev = 0u;
            in = inv;
            if (p.boxes) {
                const int box = i % p.boxes;
                ok = ok && mbar_wait(smem_addr(&B.words_full[box]), (i / p.boxes) & 1, stop, err);
                const unsigned char* q = boxes + (box * kRows + r) * RB + 16 + 8 * K * half;
#pragma unroll
                for (int h = 0; h < 2 * K; h += 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(q + 4 * h);
                    words[h] = v.x;
                    words[h + 1] = v.y;
                }
                prev = *reinterpret_cast<const uint32_t*>(q - 4);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&B.words_empty[box]));
            } else {
#pragma unroll
                for (int h = 0; h < 2 * K; ++h) words[h] = 0u;
                if (in_row) {
                    const uint32_t* q = bits + c / 32 * K;
                    load_words<K>(q, words, wide);
                    if (!first) prev = __ldg(q - 1);
                }
            }
            if (in_row) {
                if (first) prev = __ldg(w.start_state + row * nb + j);
                sc = w.scale ? __ldg(w.scale + row * nb + j) : 1.f;
            }
        };
        uint32_t words[2 * K], prev;
        float sc, pw;
        long long u = u0 + group;
        if (u < u1) fetch(group, words, prev, sc, pw);
        int done = 0;
        for (long long s0 = u0; s0 < u1 && ok; ++done) {  // segments: runs of one tile's units
            const long long seg_tile = s0 / p.steps;
            const long long s1 = (seg_tile + 1) * p.steps < u1 ? (seg_tile + 1) * p.steps : u1;
            for (; u < s1; u += 2) {
                const int it = 2 * (int)(u - u0);  // the unit's first stage
                // Where the unit's stages go.  A barrier's parity tells two neighbouring phases
                // apart.  With four or more stages the wait one turn ago puts this one's
                // phase next; with two, the group must first see the other group's fill.
                // The slot is usually free by now: asked here, the answer is there after the
                // decoding, while an answer waited for takes hundreds of cycles in the queue
                // of the look-ups.
                const int step = (it + half) / p.per, sub = (it + half) % p.per;
                const int slot = step % p.slots, round = step / p.slots;
                const uint32_t empty = smem_addr(&B.empty[slot]);
                const bool ready = p.per == 2 && mbar_test(empty, (round & 1) ^ 1);
                uint32_t nwords[2 * K], nprev;
                float nsc, npw;
                if (u + 2 < u1) {
                    advance(2);
                    fetch((int)(u - u0) + 2, nwords, nprev, nsc, npw);
                }
                uint32_t v[32];
                decode_64<K, CODE>(words, prev, mask, sm, sc * inverse_pow2(pw), v);
                if (!__all_sync(0xffffffffu, ready && ok)) {
                    if (ok && p.per == 1) ok = wait_count(&B.fills[slot], kDecodeWarps / 2 * round, stop, err);
                    ok = ok && mbar_wait(empty, (round & 1) ^ 1, stop, err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
                unsigned char* a = ring + (size_t)slot * sbytes + sub * kABytes + r * 128;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4*>(a + ((q ^ (r & 7)) << 4)) =
                        make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0 || (p.per == 1 && lane == 16)) {
                    mbar_arrive(smem_addr(&B.full[slot]));
                    if (p.per == 1) atomicAdd(&B.fills[slot], 1);
                }
#pragma unroll
                for (int i = 0; i < 2 * K; ++i) words[i] = nwords[i];
                prev = nprev;
                sc = nsc;
                pw = npw;
            }
            if (!ok) break;
            // the segment's sums: lane = row, 16 tokens at a time shared among the warps
            const int acc = done & 1;
            ok = mbar_wait(smem_addr(&B.tfull[acc]), (done >> 1) & 1, stop, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const int piece = (int)blockIdx.x - cta_of(p, seg_tile * p.steps);
            float* out = partial + ((seg_tile * p.pieces + piece) * p.np) * kRows + (warp & 3) * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + acc * acc_columns;
            for (int c = 16 * (warp >> 2); c < p.np; c += 64) {
                float d[16];
                tmem_load16(lanes + c, d);
#pragma unroll
                for (int i = 0; i < 16; ++i) __stcg(out + (long long)(c + i) * kRows, d[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.tempty[acc]));
            s0 = s1;
        }
    } else if (warp == kDecodeWarps) {
        if (lane == 0) {
            bool ok = true;
            int i = 0;
            const int fills = 2 / p.per * (int)(u1 - u0);
            long long tile = u0 / p.steps;
            int ks = 2 * (int)(u0 - tile * p.steps);  // in stages
            for (; i < fills; ++i) {
                const int slot = i % p.slots;
                const uint32_t full = smem_addr(&B.full[slot]);
                ok = mbar_wait(smem_addr(&B.empty[slot]), ((i / p.slots) & 1) ^ 1, stop, err);
                if (!ok) break;
                mbar_expect_tx(full, p.per * bbytes);
                for (int h = 0; h < p.per; ++h)
                    tma_load_2d(smem_addr(ring + (size_t)slot * sbytes + p.per * kABytes + h * bbytes), &map_x, full,
                                (ks + h) * kDepth, (int)(tile / p.row_tiles) * p.np);
                ks += p.per;
                if (ks == 2 * p.steps) {
                    ks = 0;
                    ++tile;
                }
            }
            if (!ok)  // what was loaded last is still waited for (unless its decoders stopped)
                for (int j = i > p.slots ? i - p.slots : 0; j < i; ++j)
                    mbar_drain(smem_addr(&B.full[j % p.slots]), (j / p.slots) & 1);
        }
        __syncwarp();
    } else if (warp == kDecodeWarps + 2) {
        if (lane == 0 && p.boxes) {
            bool ok = true;
            int i = 0;
            const int n = (int)(u1 - u0);
            long long tile = u0 / p.steps;
            int ks = (int)(u0 - tile * p.steps);
            for (; i < n; ++i) {
                const int box = i % p.boxes;
                const uint32_t full = smem_addr(&B.words_full[box]);
                ok = mbar_wait(smem_addr(&B.words_empty[box]), ((i / p.boxes) & 1) ^ 1, stop, err);
                if (!ok) break;
                mbar_expect_tx(full, kRows * RB);
                // 16 k bytes per unit: every copy starts on a 16-byte boundary; before a row's
                // first word and behind its last the box is filled with zeros
                tma_load_2d(smem_addr(boxes + box * kRows * RB), &map_words, full, 4 * K * ks - 4,
                            (int)(tile % p.row_tiles) * kRows);
                if (++ks == p.steps) {
                    ks = 0;
                    ++tile;
                }
            }
            if (!ok)
                for (int j = i > p.boxes ? i - p.boxes : 0; j < i; ++j)
                    mbar_drain(smem_addr(&B.words_full[j % p.boxes]), (j / p.boxes) & 1);
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            const uint32_t idesc = mma_idesc(kRows, p.np, 0, 0, 0);
            const unsigned long long desc0 = smem_desc_sw128(smem_addr(ring), 16);
            bool ok = true;
            int done = 0;
            for (long long s0 = u0; s0 < u1 && ok; ++done) {
                const long long tile = s0 / p.steps;
                const long long s1 = (tile + 1) * p.steps < u1 ? (tile + 1) * p.steps : u1;
                const int acc = done & 1;
                ok = mbar_wait(smem_addr(&B.tempty[acc]), ((done >> 1) & 1) ^ 1, stop, err);
                if (!ok) break;
                tc_fence_after();
                const int first = 2 / p.per * (int)(s0 - u0), last = 2 / p.per * (int)(s1 - u0);
                for (int i = first; i < last; ++i) {
                    const int slot = i % p.slots;
                    ok = mbar_wait(smem_addr(&B.full[slot]), (i / p.slots) & 1, stop, err);
                    if (!ok) break;
                    tc_fence_after();
                    // descriptors count in 16 bytes
                    unsigned long long a = desc0 + (unsigned)(slot * sbytes >> 4), b = a + (unsigned)(p.per * kABytes >> 4);
                    for (int h = 0; h < p.per; ++h, a += kABytes >> 4, b += (unsigned)(bbytes >> 4)) {
#pragma unroll
                        for (int j = 0; j < kDepth / 16; ++j)
                            mma_f16<1>(tmem + acc * acc_columns, a + 2 * j, b + 2 * j, idesc,
                                       i != first || h != 0 || j != 0);
                    }
                    mma_commit<1>(smem_addr(&B.empty[slot]));
                }
                if (ok) mma_commit<1>(smem_addr(&B.tfull[acc]));
                s0 = s1;
            }
            if (!ok) {
                mma_commit<1>(smem_addr(&B.drain));
                mbar_drain(smem_addr(&B.drain), 0);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kDecodeWarps + 1) {
        tc_fence_after();
        tmem_free<1>(tmem, p.tmem_columns);
    }
}

// Adds a tile's pieces in order and applies the epilogue: a warp takes one token of a
// tile, four rows of W per lane.
template <int XT>
__global__ void __launch_bounds__(256) fused_finish_kernel(Plan p, Epilogue e, long long rows, const float* partial,
                                                           bool vec)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long tile = blockIdx.x;
    const long long t = (tile / p.row_tiles) * p.np + (long long)blockIdx.y * 8 + (threadIdx.x >> 5);
    const int local = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (local >= p.np || t >= p.n) return;
    const long long r = (tile % p.row_tiles) * kRows + 4 * lane;
    const int pieces = cta_of(p, (tile + 1) * p.steps - 1) - cta_of(p, tile * p.steps) + 1;
    const float* src = partial + (tile * p.pieces * p.np + local) * kRows + 4 * lane;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < pieces; ++i) {
        const float4 d = __ldcg(reinterpret_cast<const float4*>(src + (long long)i * p.np * kRows));
        v[0] += d.x; v[1] += d.y; v[2] += d.z; v[3] += d.w;
    }
    const int count = rows - r < 4 ? (rows - r > 0 ? (int)(rows - r) : 0) : 4;
    const float rs = e.row_scale ? __ldg(e.row_scale + t) : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] *= rs;
        if (i < count) v[i] = fmaf(v[i], e.col_scale ? __ldg(e.col_scale + r + i) : 1.f, e.bias ? __ldg(e.bias + r + i) : 0.f);
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
        if (count > 0 && (lane & 7) == 0) e.z_scales[t * ((rows + 31) / 32) + r / 32] = (uint8_t)byte;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count)
                e.z_codes[t * rows + r + i] = byte == 255u ? 0 : (uint8_t)(int8 ? q8_encode<TCQ_Q8_INT8>(v[i], inv)
                                                                              : q8_encode<TCQ_Q8_E4M3>(v[i], inv));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], e.act);
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

int code_of(const CodedMatrix& w) { return w.cb_f16 == 1 ? kCode16F16 : w.cb_f16 == 0 ? kCode16F32 : kCode16Mad; }

// `words_tma`: the stream's rows can be read by TMA
Plan make_plan(int code, int L, int K, long long rows, long long cols, long long n, int num_sms, bool words_tma)
{
    Plan p;
    p.n = n;
    const long long tt = (n + 255) / 256;
    p.token_tiles = (int)tt;
    p.np = (int)(((n + tt - 1) / tt + 15) / 16 * 16);
    p.row_tiles = (int)((rows + kRows - 1) / kRows);
    p.steps = (int)((cols + 127) / 128);
    p.units = (long long)p.row_tiles * p.token_tiles * p.steps;
    // at least two units per CTA, one for each group of decoding warps
    long long ctas = (p.units + 1) / 2;
    if (ctas > num_sms) ctas = num_sms;
    p.ctas = (int)ctas;
    const long long least = p.units / p.ctas;  // a tile meets at most this many CTAs
    p.pieces = (int)((p.steps + least - 1) / least + 1);
    if (p.pieces > p.ctas) p.pieces = p.ctas;
    p.table = (int)((table_bytes(code, L) + 1023) & ~(size_t)1023);
    // slots of a whole unit, one barrier and one commit for 128 columns, where two of them
    // fit beside the table (the barriers of a slot share the pipe that the look-ups fill,
    // about 300 cycles each); slots of a stage otherwise
    const int room = kSmemBytes - p.table - (int)sizeof(Barriers), stage = kABytes + p.np * kDepth * 2;
    const int box = kRows * box_row_bytes(K);
    p.per = room >= 4 * stage ? 2 : 1;
    p.slots = p.per == 2 ? (room - (words_tma ? kMaxBoxes * box : 0)) / (2 * stage) : 2;
    if (p.slots < 2) p.slots = 2;
    if (p.slots > kMaxSlots) p.slots = kMaxSlots;
    p.boxes = words_tma ? (room - p.slots * p.per * stage) / box : 0;
    // an even number, so that a group's boxes are its own: it has then seen the phase before
    p.boxes = p.boxes >= kMaxBoxes ? kMaxBoxes : p.boxes / 2 * 2;
    p.tmem_columns = 32;
    while (p.tmem_columns < 2 * p.np) p.tmem_columns *= 2;
    return p;
}

template <int K, int CODE>
cudaError_t launch(const CodedMatrix& w, const CUtensorMap& map, const CUtensorMap& words, const Plan& p, const float* row_pow2, float* partial,
                   unsigned int* err, bool early, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(fused_kernel<K, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemBytes);
    if (e != cudaSuccess) return e;
    const size_t smem = p.table + (size_t)p.slots * p.per * (kABytes + p.np * kDepth * 2) + p.boxes * kRows * box_row_bytes(K) +
                        sizeof(Barriers);
    return launch_pdl(fused_kernel<K, CODE>, dim3(p.ctas), dim3(kThreads), smem, stream, early, w, map, words, p, row_pow2,
                      partial, err);
}

template <int CODE>
cudaError_t launch_k(const CodedMatrix& w, const CUtensorMap& map, const CUtensorMap& words, const Plan& p, const float* row_pow2, float* partial,
                     unsigned int* err, bool early, cudaStream_t stream)
{
    switch (w.K) {
    case 1: return launch<1, CODE>(w, map, words, p, row_pow2, partial, err, early, stream);
    case 2: return launch<2, CODE>(w, map, words, p, row_pow2, partial, err, early, stream);
    case 3: return launch<3, CODE>(w, map, words, p, row_pow2, partial, err, early, stream);
    default: return launch<4, CODE>(w, map, words, p, row_pow2, partial, err, early, stream);
    }
}

}  // namespace

// T a multiple of 64 keeps a stage inside one block and its words together.
bool fused_shape(int T, long long rows, long long cols, long long n)
{
    return T % kDepth == 0 && n <= kFusedMaxTokens && (rows / kRows + 1) * ((n + 255) / 256) * (cols / 128 + 1) < (1ll << 30);
}

size_t fused_partial_bytes(int cb_f16, int L, long long rows, long long cols, long long n, int num_sms)
{
    const int code = cb_f16 == 1 ? kCode16F16 : cb_f16 == 0 ? kCode16F32 : kCode16Mad;
    const Plan p = make_plan(code, L, 1, rows, cols, n, num_sms, false);  // the pieces do not depend on the ring
    return (size_t)p.row_tiles * p.token_tiles * p.pieces * p.np * kRows * sizeof(float);
}

cudaError_t launch_gemm_fused(const CodedMatrix& w, const void* x, long long ldx, long long n, int xdtype,
                              const float* row_pow2, float* partial, const Epilogue& e, int num_sms, unsigned int* err,
                              bool early, cudaStream_t stream)
{
    const int code = code_of(w);
    const long long row_words = w.cols / 32 * w.K;
    const bool words_tma = (reinterpret_cast<uintptr_t>(w.bits) & 15) == 0 && row_words % 4 == 0;
    const Plan p = make_plan(code, w.L, w.K, w.rows, w.cols, n, num_sms, words_tma);
    CUtensorMap map, words;
    if (!make_map_16bit(&map, x, n, w.cols, ldx, p.np)) return cudaErrorInvalidValue;
    if (p.boxes == 0)
        words = map;  // not used
    else if (!make_map_words(&words, w.bits, w.rows, row_words, 4 * (w.K + 1), kRows))
        return cudaErrorInvalidValue;
    cudaError_t st = code == kCode16Mad   ? launch_k<kCode16Mad>(w, map, words, p, row_pow2, partial, err, early, stream)
                     : code == kCode16F16 ? launch_k<kCode16F16>(w, map, words, p, row_pow2, partial, err, early, stream)
                                          : launch_k<kCode16F32>(w, map, words, p, row_pow2, partial, err, early, stream);
    if (st != cudaSuccess) return st;
    bool vec = (reinterpret_cast<uintptr_t>(e.out) & 7) == 0 && e.ldo % 4 == 0;
    if (e.residual) vec = vec && (reinterpret_cast<uintptr_t>(e.residual) & 7) == 0 && e.ldr % 4 == 0;
    const dim3 grid((unsigned)(p.row_tiles * p.token_tiles), (unsigned)((p.np + 7) / 8));
    return launch_pdl(xdtype == TCQ_X_BF16 ? fused_finish_kernel<TCQ_X_BF16> : fused_finish_kernel<TCQ_X_F16>, grid,
                      dim3(256), 0, stream, true, p, e, w.rows, static_cast<const float*>(partial), vec);
}

}  // namespace tcq
