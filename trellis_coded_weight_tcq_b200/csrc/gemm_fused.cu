// gemm_fused.cu -- the forward product for small batches: the matrix is decoded
// inside the product and never written out.
//
// With few tokens the product is bound by decoding (one shared-memory lookup per
// weight, about 3.5 bank passes per 32 random entries), so every weight is decoded
// once and goes straight into a tensor-core operand tile.  The
// weights take the M side of the MMA: a CTA multiplies 128 rows of W by up to 256
// tokens, D[row, token] in tensor memory (cta_group::1, 128 x N x 16).
//
// 16 warps decode, in two groups that take turns at units of 128 columns (two stages
// of the ring): a warp covers 16 rows, lanes 0-15 the first stage's 64 columns of
// them, lanes 16-31 the second's.  A lane turns its 2 k stream words into eight 16-byte
// pieces of the swizzled K-major tile, held in registers until the stage is free.
// The look-ups leave the load/store pipe little room (46k of the kernel's 90k cycles for
// 14336 x 4096), so the stream words come by TMA where shared memory and their alignment
// allow: a box of 128 rows by a unit's words and the four before them per group; a warp's
// reads of 16 separate rows from global memory would take 16 passes each.  Otherwise a
// warp reads whole 32-byte sectors of its rows.  Warp 16 loads the activations' tiles,
// warp 18 the stream words, one thread of warp 17 issues the MMAs.
//
// Measured on a B200, 14336 x 4096, L = 16, k = 2, bfloat16: 53 us for 24 tokens and 76 us
// for 200, of which the pass before (the activations' and the matrix's powers) and the
// pieces' sums after it take 6 and 6 us alone (the look-ups: 24 us; 24 and 200 tokens' MMAs: 2
// and 14 us).  Writing the matrix out first (38 us) and multiplying it takes 81 and 84 us.
//
// Work is split over the SMs evenly, in units: a CTA takes a contiguous run of (tile,
// unit) pairs, so a tile's reduction may be cut into pieces; each writes its fp32 sums
// to the workspace, and a second kernel adds a tile's pieces in order and applies the
// epilogue.  The split depends on the shape and the SM count only.
#include "decode16.cuh"
#include "epilogue.cuh"
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
constexpr int kSlots = 2;              // of the operand ring
constexpr int kSmemBytes = 227 * 1024;

struct Barriers {
    unsigned long long full[kSlots], empty[kSlots], tfull[2], tempty[2], drain;
    unsigned long long go[2];           // a group may decode its next unit
    unsigned long long words_empty[2];  // a group has read its box of stream words
    uint32_t tmem;
    int stop;
    int fills[kSlots];  // warps that have filled a slot, counted from the start
    uint32_t tops[kThreads / 32];  // of the table (staged_table_power)
};

struct Plan {
    long long n;          // tokens, at most 256
    int np;               // n rounded up to a multiple of 16
    int row_tiles;
    int steps;            // units of 128 columns of a whole reduction
    long long units;      // tiles * steps
    int ctas;
    int pieces;           // slots per tile in the workspace
    int per;              // stages per slot: 2 (a unit), or 1 where only two stages fit
    int tmem_columns;
    int table;            // shared-memory bytes of the table, a multiple of 1024
    int boxes;            // 1: a box of stream words per group, 0: words from global memory
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

// The same from a box in shared memory (8 k bytes, aligned to 8, for even k to 16).
template <int K>
__device__ __forceinline__ void read_words(const unsigned char* p, uint32_t (&w)[2 * K])
{
    if constexpr (K % 2 == 0) {
#pragma unroll
        for (int i = 0; i < 2 * K; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2 * K; i += 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * i);
            w[i] = v.x; w[i + 1] = v.y;
        }
    }
}

template <int K, int CODE>
__global__ void __launch_bounds__(kThreads, 1)
fused_kernel(CodedMatrix w, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_words,
             Plan p, WeightPowers powers, float* partial, unsigned int* err)
{
    constexpr int RB = box_row_bytes(K);
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* ring = sm + p.table;
    const int bbytes = p.np * kDepth * 2;
    const int sbytes = p.per * (kABytes + bbytes);  // a slot: its A stages, then its B stages
    unsigned char* boxes = ring + kSlots * sbytes;
    Barriers& B = *reinterpret_cast<Barriers*>(boxes + 2 * p.boxes * kRows * RB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&B.full[i]), kDecodeWarps / 2 + 1);  // a group's warps, and the TMA thread
            mbar_init(smem_addr(&B.empty[i]), 1);
            B.fills[i] = 0;
            mbar_init(smem_addr(&B.tfull[i]), 1);
            mbar_init(smem_addr(&B.tempty[i]), kDecodeWarps);
            // the other group has decoded its unit before, the words are there, the slot is free
            mbar_init(smem_addr(&B.go[i]), kDecodeWarps / 2 + p.boxes + (p.per == 2));
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
    float table = 1.f;  // the table's power
    if constexpr (CODE == kCode16F32) {
        // written ahead of the wait below: a launch that starts early follows one of this call's,
        // which began after whatever used the workspace before
        if (powers.staged) table = staged_table_power(reinterpret_cast<const float*>(sm), 1 << w.L, B.tops, powers.table_out);
    }
    pdl_wait();  // the scaled activations and the weights' powers
    pdl_release();
    const TableParts parts(CODE == kCode16F16 ? powers.table : nullptr);
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
        // where the next unit is: its tile, its place in the reduction, this lane's row
        long long tile = u0 / p.steps;
        int ks = (int)(u0 - tile * p.steps);
        const uint32_t *bits = nullptr, *start = nullptr;  // of the row, or none
        const float* scale = nullptr;
        float inv = 1.f;  // the row's power
        auto enter_tile = [&]() {
            const long long row = tile * kRows + r;
            bits = row < w.rows ? w.bits + row * (cols / 32 * K) : nullptr;
            start = w.start_state + row * nb;
            scale = w.scale ? w.scale + row * nb : nullptr;
            if (bits && scale && TCQ_IN_BOUNDS(row, w.rows)) inv = __ldcg(powers.row + row);
        };
        auto advance = [&](int by) {
            for (ks += by; ks >= p.steps; ks -= p.steps) {
                ++tile;
                if (ks - p.steps < p.steps) enter_tile();
            }
        };
        enter_tile();
        advance(group);
        // What the next unit needs from global memory, on its way while this one is decoded:
        // its block's start state where the lane's columns begin one, its scale, the row's
        // power, and without the ring of boxes its words and the one before them.
        uint32_t nwords[2 * K], nprev = 0u;
        float nsc = 0.f, npw = 1.f;
        bool nfirst = false, nout = false;  // columns behind the last
        auto fetch = [&]() {
            const int c = ks * 128 + half * kDepth;
            const int j = tshift >= 0 ? c >> tshift : c / T;
            nfirst = c == j * T;
            nout = c >= cols;
            nsc = 0.f;
            nprev = 0u;
            npw = inv;
            if (!p.boxes) {
#pragma unroll
                for (int h = 0; h < 2 * K; ++h) nwords[h] = 0u;
            }
            if (bits && c < cols && TCQ_IN_BOUNDS(bits - w.bits + c / 32 * K + 2 * K - 1, w.rows * (cols / 32 * K)) &&
                TCQ_IN_BOUNDS(start - w.start_state + j, w.rows * nb)) {
                if (!p.boxes) load_words<K>(bits + c / 32 * K, nwords, wide);
                if (nfirst)
                    nprev = __ldg(start + j);
                else if (!p.boxes)
                    nprev = __ldg(bits + c / 32 * K - 1);
                nsc = scale ? __ldg(scale + j) : 1.f;
            }
        };
        bool ok = true;
        long long u = u0 + group;
        if (u < u1) fetch();
        if constexpr (CODE == kCode16F16) table = parts.power();
        // Slots of a unit belong to a group each, slots of a stage to a half of every unit.
        const int slot = p.per == 2 ? group : half;
        const uint32_t go = smem_addr(&B.go[group]);
        if (group == 1 && lane == 0) mbar_arrive(smem_addr(&B.go[0]));  // there is no unit before the first
        const unsigned char* box = boxes + (group * kRows + r) * RB + 16 + 8 * K * half;
        unsigned char* const a = ring + slot * sbytes + (p.per == 2 ? half * kABytes : 0) + r * 128;
        int own = 0;  // the group's units so far
        int done = 0;
        // A segment's sums are written after the group's first unit of the next one, while the
        // other group decodes: lane = row, 16 tokens at a time shared among the warps.
        long long pending = -1;
        int pending_set = 0, pending_parity = 0;
        auto flush = [&]() {
            if (pending < 0 || !ok) return;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&B.tfull[pending_set]), pending_parity, stop, err));
            if (!ok) return;
            tc_fence_after();
            const int piece = (int)blockIdx.x - cta_of(p, pending * p.steps);
            float* out = partial + ((pending * p.pieces + piece) * p.np) * kRows + (warp & 3) * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + pending_set * acc_columns;
            for (int c = 16 * (warp >> 2); c < p.np; c += 64) {
                float d[16];
                tmem_load16(lanes + c, d);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (TCQ_IN_BOUNDS(out - partial + (long long)(c + i) * kRows, (long long)p.row_tiles * p.pieces * p.np * kRows))
                        __stcg(out + (long long)(c + i) * kRows, d[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&B.tempty[pending_set]));
            pending = -1;
        };
        for (long long s0 = u0; s0 < u1 && ok; ++done) {  // segments: runs of one tile's units
            const long long seg_tile = s0 / p.steps;
            const long long s1 = (seg_tile + 1) * p.steps < u1 ? (seg_tile + 1) * p.steps : u1;
            for (; u < s1; u += 2, ++own) {
                uint32_t words[2 * K], prev = nprev;
                const float sc = nsc, pw = npw;
                const bool first = nfirst, out = nout;
#pragma unroll
                for (int h = 0; h < 2 * K; ++h) words[h] = nwords[h];
                if (u + 2 < u1) {
                    advance(2);
                    fetch();
                }
                // The groups decode in turns: one fills the load/store pipe by itself, and the
                // other stores, fetches and waits meanwhile (left alone they fall into step).
                // A wait takes hundreds of cycles in the queue of the other's look-ups, so
                // one barrier stands for all that a unit needs.
                ok = ok && mbar_wait(go, own & 1, stop, err);
                if (p.boxes) {
                    read_words<K>(box, words);
                    const uint32_t before = *reinterpret_cast<const uint32_t*>(box - 4);
                    if (!first) prev = before;
                }
                uint32_t v[32];
                decode_64<K, CODE>(words, prev, mask, sm, sc * inverse_pow2(power_product(pw, table)), v);
                if (out) {  // no weight: entry 0 need not be finite, and 0 times it would spoil the row
#pragma unroll
                    for (int h = 0; h < 32; ++h) v[h] = 0u;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_addr(&B.go[group ^ 1]));
                    if (p.boxes) mbar_arrive(smem_addr(&B.words_empty[group]));
                }
                if (p.per == 1) {
                    // A barrier's parity tells two neighbouring phases apart: the group must
                    // first see the other group's fill of these slots.
                    const int round = 2 * own + group;
                    ok = ok && wait_count(&B.fills[slot], kDecodeWarps / 2 * round, stop, err) &&
                         mbar_wait(smem_addr(&B.empty[slot]), (round & 1) ^ 1, stop, err);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4*>(a + ((q ^ (r & 7)) << 4)) =
                        make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                fence_async_shared();
                __syncwarp();
                if (lane == 0 || (p.per == 1 && lane == 16)) {
                    mbar_arrive(smem_addr(&B.full[slot]));
                    if (p.per == 1) atomicAdd(&B.fills[slot], 1);
                }
                if (pending >= 0) flush();
            }
            if (!ok) break;
            flush();  // of the segment before, where the group had no unit in this one
            pending = seg_tile;
            pending_set = done & 1;
            pending_parity = (done >> 1) & 1;
            s0 = s1;
        }
        flush();
    } else if (warp == kDecodeWarps) {
        if (lane == 0) {
            bool ok = true;
            int i = 0;
            const int fills = 2 / p.per * (int)(u1 - u0);
            long long tile = u0 / p.steps;
            int ks = 2 * (int)(u0 - tile * p.steps);  // in stages
            for (; i < fills; ++i) {
                const int slot = i & 1;
                const uint32_t full = smem_addr(&B.full[slot]);
                ok = mbar_wait(smem_addr(&B.empty[slot]), ((i >> 1) & 1) ^ 1, stop, err);
                if (!ok) break;
                mbar_expect_tx(full, p.per * bbytes);
                for (int h = 0; h < p.per; ++h)
                    tma_load_2d(smem_addr(ring + slot * sbytes + p.per * kABytes + h * bbytes), &map_x, full,
                                (ks + h) * kDepth, 0);
                ks += p.per;
                if (ks == 2 * p.steps) {
                    ks = 0;
                    ++tile;
                }
            }
            if (!ok)  // what was loaded last is still waited for (unless its decoders stopped)
                for (int j = i > kSlots ? i - kSlots : 0; j < i; ++j) mbar_drain(smem_addr(&B.full[j & 1]), (j >> 1) & 1);
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
                const int g = i & 1;
                const uint32_t go = smem_addr(&B.go[g]);
                ok = mbar_wait(smem_addr(&B.words_empty[g]), ((i >> 1) & 1) ^ 1, stop, err);
                if (!ok) break;
                mbar_expect_tx(go, kRows * RB);
                // 16 k bytes per unit: every copy starts on a 16-byte boundary; before a row's
                // first word and behind its last the box is filled with zeros
                tma_load_2d(smem_addr(boxes + g * kRows * RB), &map_words, go, 4 * K * ks - 4,
                            (int)tile * kRows);
                if (++ks == p.steps) {
                    ks = 0;
                    ++tile;
                }
            }
            if (!ok)
                for (int j = i > 2 ? i - 2 : 0; j < i; ++j) mbar_drain(smem_addr(&B.go[j & 1]), (j >> 1) & 1);
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            const uint32_t idesc = mma_idesc(kRows, p.np, 0, 0, 0);
            const unsigned long long desc0 = smem_desc_sw128(smem_addr(ring), 16);
            bool ok = true;
            int done = 0;
            if (p.per == 2)  // both slots start free
                for (int g = 0; g < 2; ++g) mbar_arrive(smem_addr(&B.go[g]));
            for (long long s0 = u0; s0 < u1 && ok; ++done) {
                const long long tile = s0 / p.steps;
                const long long s1 = (tile + 1) * p.steps < u1 ? (tile + 1) * p.steps : u1;
                const int acc = done & 1;
                ok = mbar_wait(smem_addr(&B.tempty[acc]), ((done >> 1) & 1) ^ 1, stop, err);
                if (!ok) break;
                tc_fence_after();
                const int first = 2 / p.per * (int)(s0 - u0), last = 2 / p.per * (int)(s1 - u0);
                for (int i = first; i < last; ++i) {
                    const int slot = i & 1;
                    ok = mbar_wait(smem_addr(&B.full[slot]), (i >> 1) & 1, stop, err);
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
                    if (p.per == 2) mma_commit<1>(smem_addr(&B.go[slot]));
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
    const int t = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (t >= p.n) return;
    const long long r = tile * kRows + 4 * lane;
    const int pieces = cta_of(p, (tile + 1) * p.steps - 1) - cta_of(p, tile * p.steps) + 1;
    const float* src = partial + (tile * p.pieces * p.np + t) * kRows + 4 * lane;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
        if (!TCQ_IN_BOUNDS(src - partial + (long long)i * p.np * kRows + 3, (long long)p.row_tiles * p.pieces * p.np * kRows))
            break;
        const float4 d = __ldcg(reinterpret_cast<const float4*>(src + (long long)i * p.np * kRows));
        v[0] += d.x; v[1] += d.y; v[2] += d.z; v[3] += d.w;
    }
    finish_quad<XT>(e, t, r, p.n, rows, v, vec);
}

int code_of(const CodedMatrix& w) { return w.cb_f16 == 1 ? kCode16F16 : w.cb_f16 == 0 ? kCode16F32 : kCode16Mad; }

// `words_tma`: the stream's rows can be read by TMA
Plan make_plan(int code, int L, int K, long long rows, long long cols, long long n, int num_sms, bool words_tma)
{
    Plan p;
    p.n = n;
    p.np = (int)((n + 15) / 16 * 16);
    p.row_tiles = (int)((rows + kRows - 1) / kRows);
    p.steps = (int)((cols + 127) / 128);
    p.units = (long long)p.row_tiles * p.steps;
    // two units per CTA at least, one for each group of decoding warps (of an odd number of
    // units one CTA may get a single one, and its second group none)
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
    p.boxes = words_tma && room - kSlots * p.per * stage >= 2 * box;
    p.tmem_columns = 32;
    while (p.tmem_columns < 2 * p.np) p.tmem_columns *= 2;
    return p;
}

template <int K, int CODE>
cudaError_t launch(const CodedMatrix& w, const CUtensorMap& map, const CUtensorMap& words, const Plan& p,
                   const WeightPowers& powers, float* partial, unsigned int* err, bool early, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(fused_kernel<K, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemBytes);
    if (e != cudaSuccess) return e;
    const size_t smem = p.table + (size_t)kSlots * p.per * (kABytes + p.np * kDepth * 2) +
                        2 * p.boxes * kRows * box_row_bytes(K) + sizeof(Barriers);
    return launch_pdl(fused_kernel<K, CODE>, dim3(p.ctas), dim3(kThreads), smem, stream, early, w, map, words, p, powers,
                      partial, err);
}

template <int CODE>
cudaError_t launch_k(const CodedMatrix& w, const CUtensorMap& map, const CUtensorMap& words, const Plan& p,
                     const WeightPowers& powers, float* partial, unsigned int* err, bool early, cudaStream_t stream)
{
    switch (w.K) {
    case 1: return launch<1, CODE>(w, map, words, p, powers, partial, err, early, stream);
    case 2: return launch<2, CODE>(w, map, words, p, powers, partial, err, early, stream);
    case 3: return launch<3, CODE>(w, map, words, p, powers, partial, err, early, stream);
    default: return launch<4, CODE>(w, map, words, p, powers, partial, err, early, stream);
    }
}

}  // namespace

// T a multiple of 64 keeps a stage inside one block and its words together.  More than
// 256 tokens would decode the matrix again, and the product that decodes ahead wins.
// Measured, here / decoded ahead, in us (bfloat16, binary16 table, scales): 14336 x 4096 32
// tokens 53 / 78, 192 75 / 82, 256 84 / 84; 4096 x 14336 32 tokens 55 / 77, 256 76 / 84;
// 4096 x 4096 32 tokens 26 / 31, 256 35 / 38; 512 x 512 32 tokens 13 / 18, 256 18 / 18.
// Nor does this one need room for the matrix in 16 bits.
bool fused_shape(int T, long long rows, long long cols, long long n)
{
    return T % kDepth == 0 && n <= 256 && (rows / kRows + 1) * (cols / 128 + 1) < (1ll << 30);
}

size_t fused_partial_bytes(int cb_f16, int L, long long rows, long long cols, long long n, int num_sms)
{
    const int code = cb_f16 == 1 ? kCode16F16 : cb_f16 == 0 ? kCode16F32 : kCode16Mad;
    const Plan p = make_plan(code, L, 1, rows, cols, n, num_sms, false);  // the pieces do not depend on the ring
    return (size_t)p.row_tiles * p.pieces * p.np * kRows * sizeof(float);
}

cudaError_t launch_gemm_fused(const CodedMatrix& w, const void* x, long long ldx, long long n, int xdtype,
                              const WeightPowers& powers, float* partial, const Epilogue& e, int num_sms, unsigned int* err,
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
    cudaError_t st = code == kCode16Mad   ? launch_k<kCode16Mad>(w, map, words, p, powers, partial, err, early, stream)
                     : code == kCode16F16 ? launch_k<kCode16F16>(w, map, words, p, powers, partial, err, early, stream)
                                          : launch_k<kCode16F32>(w, map, words, p, powers, partial, err, early, stream);
    if (st != cudaSuccess) return st;
    bool vec = (reinterpret_cast<uintptr_t>(e.out) & 7) == 0 && e.ldo % 4 == 0;
    if (e.residual) vec = vec && (reinterpret_cast<uintptr_t>(e.residual) & 7) == 0 && e.ldr % 4 == 0;
    const dim3 grid((unsigned)p.row_tiles, (unsigned)((p.np + 7) / 8));
    return launch_pdl(xdtype == TCQ_X_BF16 ? fused_finish_kernel<TCQ_X_BF16> : fused_finish_kernel<TCQ_X_F16>, grid,
                      dim3(256), 0, stream, true, p, e, w.rows, static_cast<const float*>(partial), vec);
}

}  // namespace tcq
