// decode16.cu -- a trellis-coded matrix written out in 16 bits, the operand of the
// tensor-core products for batches too large to decode inside the product.
//
// A weight is scale * c[s], rounded once to binary16.  So that small scales do not
// fall into binary16's subnormals, every row is divided by a power of two, the
// least above its largest finite |scale|, and tables by one of their own, so that
// their largest entry ends in [2^14, 2^15) (the computed code's numbers too): a weight is then below 2^15, and what a
// row's largest weight is to its others, not how large they are, decides what they
// lose.  The products multiply the powers back in (exactly).  Without scales a
// binary16 or computed codeword is stored as it is.  For large bfloat16 batches the weights are
// rounded once to bfloat16 instead, as they are: its range needs no powers.
//
// A warp takes 256 columns of a row at a time, eight per lane: their windows lie in
// two stream words, one 16-byte store per lane; each warp has a contiguous run.  Table
// lookups at random shared-memory addresses bound it (as in the decoder, about 3.6 bank
// passes per 32), then the 2 bytes per weight written: 39 us for 14336 x 4096, L = 16,
// k = 2 (the look-ups alone 24 us, the 132 MB read and written 21 us).
#include "codes.cuh"
#include "decode16.cuh"
#include "gemm.cuh"
#include "pdl.cuh"

namespace tcq {

namespace {

constexpr int kThreads = 768;  // leaves registers for the pass over the activations, which runs beside it
constexpr int kUnit = 256;  // columns per warp step
constexpr int kAhead = 4;   // steps whose words are loaded together

// The table's power in a decoding kernel, whose table is staged (the caller has synchronised).
template <int CODE, bool BF16>
__device__ __forceinline__ float power_of_table(const WeightPowers& powers, const unsigned char* sm, int L)
{
    if constexpr (BF16 || CODE == kCode16Mad) return 1.f;
    if constexpr (CODE == kCode16F32) {
        __shared__ uint32_t warps[kThreads / 32];
        return powers.staged ? staged_table_power(reinterpret_cast<const float*>(sm), 1 << L, warps, powers.table_out) : 1.f;
    }
    return table_power(powers.table);
}

// Blocks of whole 32s: a row's stream words follow one another without gaps, so a lane's
// words lie 8 k apart from unit to unit and its window offset never changes.  The next
// four units' words load while the current four are decoded.
template <int K, int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) decode16_rows_kernel(CodedMatrix w, uint16_t* out, long long ldw,
                                                                    WeightPowers powers)
{
    extern __shared__ __align__(16) unsigned char sm[];
    stage_table<CODE>(sm, w.cb, w.cb_f16, w.L);
    pdl_wait();     // the powers
    pdl_release();  // the pass over the activations may run beside this one (and read the powers)
    const int lane = threadIdx.x & 31;
    const int cols = (int)w.cols, T = w.T, nb = cols / T;
    const int upr = (cols + kUnit - 1) / kUnit;
    const long long units = upr * w.rows;
    const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
    const long long me = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const uint32_t mask = (1u << w.L) - 1u;
    const int tshift = (T & (T - 1)) == 0 ? __ffs(T) - 1 : -1;
    const long long u0 = units * me / nwarps;
    int left = (int)(units * (me + 1) / nwarps - u0);
    long long row = u0 / upr;
    int at = (int)(u0 - row * upr);
    const int word = ((8 * lane + 8) * K - 1) >> 5;  // the last window's word in a unit
    const int down = bits_behind((8 * lane + 8) * K);
    __syncthreads();
    const float table = power_of_table<CODE, BF16>(powers, sm, w.L);
    struct Four {
        uint32_t hi[kAhead], lo[kAhead];
        float sc[kAhead];
    };
    // units at .. at + kAhead - 1 of a row
    auto fetch = [&](Four& f, long long r, int a) {
        const uint32_t* p = w.bits + r * (cols / 32 * K) + word;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int c = (a + i) * kUnit + 8 * lane;
            f.hi[i] = f.lo[i] = 0u;
            f.sc[i] = 0.f;
            if (c < cols && TCQ_IN_BOUNDS(r * (cols / 32 * K) + word + (a + i) * 8 * K, w.rows * (cols / 32 * K))) {
                const int j = tshift >= 0 ? c >> tshift : (int)((unsigned)c / (unsigned)T);
                const int e = (a + i) * 8 * K;
                f.lo[i] = __ldg(p + e);
                f.hi[i] = __ldg((c - j * T + 8) * K > 32 ? p + e - 1 : w.start_state + r * nb + j);
                f.sc[i] = w.scale ? __ldg(w.scale + r * nb + j) : 1.f;
            }
        }
    };
    Four cur, nxt;
    if (left > 0) fetch(cur, row, at);
    while (left > 0) {  // the same in every lane
        int n = upr - at < kAhead ? upr - at : kAhead;
        if (n > left) n = left;
        const long long r = row;
        const int a = at;
        at += n;
        left -= n;
        if (at == upr) {
            at = 0;
            ++row;
        }
        if (left > 0) fetch(nxt, row, at);
        const float inv = BF16 ? 1.f : inverse_pow2(power_product(powers.row ? __ldcg(powers.row + r) : 1.f, table));
        uint16_t* dst = out + r * ldw + a * kUnit + 8 * lane;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i >= n) break;
            uint32_t v[4];
            decode_weights<K, 8, CODE, BF16>(cur.hi[i], cur.lo[i], down, mask, sm, cur.sc[i] * inv, v);
            // ldw is cols rounded up to 8: a lane's eight columns are all stored or none is
            if ((a + i) * kUnit + 8 * lane < cols && TCQ_IN_BOUNDS(dst - out + i * kUnit + 7, w.rows * ldw))
                *reinterpret_cast<uint4*>(dst + i * kUnit) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        cur = nxt;
    }
}

// Any block of whole quads; N = 8: whole eights, 4: two reads per lane.
template <int K, int CODE, int N, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) decode16_kernel(CodedMatrix w, uint16_t* out, long long ldw,
                                                               WeightPowers powers)
{
    constexpr int H = 8 / N;  // reads per lane and unit
    extern __shared__ __align__(16) unsigned char sm[];
    stage_table<CODE>(sm, w.cb, w.cb_f16, w.L);
    pdl_wait();
    pdl_release();
    __syncthreads();
    const float table = power_of_table<CODE, BF16>(powers, sm, w.L);
    const int lane = threadIdx.x & 31;
    const int cols = (int)w.cols, T = w.T, W = w.W, nb = cols / T;
    const int upr = (cols + kUnit - 1) / kUnit;
    const long long units = upr * w.rows;
    const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
    const long long me = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const uint32_t mask = (1u << w.L) - 1u;
    const long long u0 = units * me / nwarps, u1 = units * (me + 1) / nwarps;
    long long row = u0 / upr;
    int at = (int)(u0 - row * upr);
    for (long long u = u0; u < u1; ++u) {
        const float inv = BF16 ? 1.f : inverse_pow2(power_product(powers.row ? __ldcg(powers.row + row) : 1.f, table));
        const int c = at * kUnit + 8 * lane;
        uint32_t v[4];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int ch = c + N * h;
            uint32_t hi = 0u, lo = 0u;
            float sc = 0.f;
            int down = 0;
            if (ch < cols) {
                const int j = (int)((unsigned)ch / (unsigned)T);
                const long long b = row * nb + j;
                const int end = (ch - j * T + N) * K;  // of the last window, in the block's stream
                down = bits_behind(end);
                if (TCQ_IN_BOUNDS(b, w.rows * nb)) {
                    const uint32_t* p = w.bits + b * W + ((end - 1) >> 5);
                    lo = __ldg(p);
                    hi = __ldg(end > 32 ? p - 1 : w.start_state + b);
                    sc = w.scale ? __ldg(w.scale + b) * inv : inv;
                }
            }
            decode_weights<K, N, CODE, BF16>(hi, lo, down, mask, sm, sc, v + N / 2 * h);
        }
        if (c < cols && TCQ_IN_BOUNDS(row * ldw + c + 7, w.rows * ldw))
            *reinterpret_cast<uint4*>(out + row * ldw + c) = make_uint4(v[0], v[1], v[2], v[3]);
        if (++at == upr) {
            at = 0;
            ++row;
        }
    }
}

template <int K, int CODE, bool BF16>
cudaError_t launch(const CodedMatrix& w, void* out, long long ldw, const WeightPowers& powers, int num_sms,
                   cudaStream_t stream)
{
    typedef void (*Kernel)(CodedMatrix, uint16_t*, long long, WeightPowers);
    const Kernel kernel = w.T % 32 == 0  ? Kernel(decode16_rows_kernel<K, CODE, BF16>)
                          : w.T % 8 == 0 ? Kernel(decode16_kernel<K, CODE, 8, BF16>)
                                         : Kernel(decode16_kernel<K, CODE, 4, BF16>);
    const size_t smem = table_bytes(CODE, w.L);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const long long units = (w.cols + kUnit - 1) / kUnit * w.rows;
    const long long need = (units + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = (int)(need < num_sms ? need : num_sms);
    return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, stream, powers.row || powers.table, w,
                      static_cast<uint16_t*>(out), ldw, powers);
}

template <int CODE, bool BF16>
cudaError_t launch_k(const CodedMatrix& w, void* out, long long ldw, const WeightPowers& powers, int num_sms,
                     cudaStream_t stream)
{
    switch (w.K) {
    case 1: return launch<1, CODE, BF16>(w, out, ldw, powers, num_sms, stream);
    case 2: return launch<2, CODE, BF16>(w, out, ldw, powers, num_sms, stream);
    case 3: return launch<3, CODE, BF16>(w, out, ldw, powers, num_sms, stream);
    default: return launch<4, CODE, BF16>(w, out, ldw, powers, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_decode16(const CodedMatrix& w, void* out, long long ldw, float* row_pow2, uint8_t* row_exponents,
                            uint32_t* table_top, int num_sms, cudaStream_t stream)
{
    // the pass over the activations, which uses the exponents, may run beside this launch
    const bool ahead = table_top && (w.cb_f16 || (w.scale && row_exponents));
    WeightPowers powers;
    if (w.scale) powers.row = row_pow2;
    powers.staged = table_top && !w.cb_f16;
    if (powers.staged && !ahead) powers.table_out = table_top;
    if (!powers.staged) powers.table = table_top;
    if (w.scale || ahead) {
        const cudaError_t e = launch_prepare({}, powers_of(w, row_pow2, row_exponents, ahead ? table_top : nullptr), stream);
        if (e != cudaSuccess) return e;
    }
    switch (w.cb_f16) {
    case kMadCodebook: return launch_k<kCode16Mad, false>(w, out, ldw, powers, num_sms, stream);
    case 1: return launch_k<kCode16F16, false>(w, out, ldw, powers, num_sms, stream);
    default: return launch_k<kCode16F32, false>(w, out, ldw, powers, num_sms, stream);
    }
}

cudaError_t launch_decode_bf16(const CodedMatrix& w, void* out, long long ldw, int num_sms, cudaStream_t stream)
{
    switch (w.cb_f16) {
    case kMadCodebook: return launch_k<kCode16Mad, true>(w, out, ldw, {}, num_sms, stream);
    case 1: return launch_k<kCode16F16, true>(w, out, ldw, {}, num_sms, stream);
    default: return launch_k<kCode16F32, true>(w, out, ldw, {}, num_sms, stream);
    }
}

}  // namespace tcq
