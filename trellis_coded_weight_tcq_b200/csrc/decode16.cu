// decode16.cu -- a trellis-coded matrix written out as binary16, the operand of
// the tensor-core products for batches too large to decode inside the product.
//
// A weight is scale * c[s], rounded once to binary16.  So that small scales do not
// fall into binary16's subnormals, every row is divided by a power of two, the
// least above its largest finite |scale|: the scales that multiply the codewords
// are then below 1 and a product never overflows where the codeword does not.  The
// products multiply the power back in (exactly).  Without scales a binary16 or
// computed codeword is stored as it is.
//
// A warp takes 256 columns of a row at a time, eight per lane: their windows lie in
// two stream words, one 16-byte store per lane; each warp has a contiguous run.  Table lookups at random
// shared-memory addresses bound it (as in the decoder), then the 2 bytes per weight
// written.
#include "codes.cuh"
#include "decode16.cuh"
#include "gemm.cuh"
#include "pdl.cuh"

namespace tcq {

namespace {

constexpr int kThreads = 768;  // leaves registers for the pass over the activations, which runs beside it
constexpr int kUnit = 256;  // columns per warp step
constexpr int kAhead = 4;   // steps whose words are loaded together

// Powers of two of the rows: one warp per row over its scales.
__global__ void __launch_bounds__(256) row_pow2_kernel(const float* scale, long long rows, long long nb, float* row_pow2)
{
    pdl_release();
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    uint32_t top = 0u;
    for (long long j = threadIdx.x & 31; j < nb; j += 32) top = max(top, finite_magnitude(__ldg(scale + r * nb + j)));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) row_pow2[r] = pow2_clamped(power_above(top));
}

// N = 8: blocks of whole eights; 4: any block of whole quads (two reads per lane).
// T32: T is a multiple of 32, so that a row's stream words follow one another without
// gaps and a lane's word index needs no division.
template <int K, int CODE, int N, bool T32>
__global__ void __launch_bounds__(kThreads, 1) decode16_kernel(CodedMatrix w, uint16_t* out, long long ldw,
                                                               const float* row_pow2)
{
    constexpr int H = 8 / N;  // reads per lane and unit
    extern __shared__ __align__(16) unsigned char sm[];
    stage_table<CODE>(sm, w.cb, w.cb_f16, w.L);
    pdl_wait();     // row_pow2
    pdl_release();  // the pass over the activations may run beside this one (and read row_pow2)
    const int lane = threadIdx.x & 31;
    const int cols = (int)w.cols, T = w.T, W = w.W, nb = cols / T;
    const int upr = (cols + kUnit - 1) / kUnit;
    const long long units = upr * w.rows;
    const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
    const long long me = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const uint32_t mask = (1u << w.L) - 1u;
    const int tshift = (T & (T - 1)) == 0 ? __ffs(T) - 1 : -1;
    // contiguous runs of units; (row, unit in the row) advance without divisions
    const long long u1 = units * (me + 1) / nwarps;
    long long u = units * me / nwarps;
    long long row = u / upr;
    int at = (int)(u - row * upr);
    const uint32_t* bits = w.bits + row * nb * W;
    const uint32_t* start = w.start_state + row * nb;
    const float* scale = w.scale ? w.scale + row * nb : nullptr;
    uint16_t* dst = out + row * ldw;
    float inv = scale && u < u1 ? inverse_pow2(__ldg(row_pow2 + row)) : 1.f;
    int left = (int)(u1 - u);
    __syncthreads();
    while (left > 0) {
        uint32_t hi[kAhead][H], lo[kAhead][H];
        float sc[kAhead][H];
        int down[kAhead][H];
        uint16_t* to[kAhead];
        const int n = left < kAhead ? left : kAhead;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i < n) {  // the same in every lane
                const int c = at * kUnit + 8 * lane;
                to[i] = c < cols ? dst + c : nullptr;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int ch = c + N * h;
                    hi[i][h] = lo[i][h] = 0u;
                    sc[i][h] = 0.f;
                    down[i][h] = 0;
                    if (ch < cols) {
                        const int j = tshift >= 0 ? ch >> tshift : (int)((unsigned)ch / (unsigned)T);
                        const int end = (ch - j * T + N) * K;  // of the last window, in the block's stream
                        const int e = T32 ? (int)(((long long)(ch + N) * K - 1) >> 5) : j * W + ((end - 1) >> 5);
                        down[i][h] = bits_behind(end);
                        if (TCQ_IN_BOUNDS((bits - w.bits) + e, w.rows * nb * W)) {
                            hi[i][h] = __ldg(end > 32 ? bits + e - 1 : start + j);
                            lo[i][h] = __ldg(bits + e);
                            sc[i][h] = scale ? __ldg(scale + j) * inv : 1.f;
                        }
                    }
                }
                if (++at == upr) {
                    at = 0;
                    ++row;
                    bits += nb * W;
                    start += nb;
                    dst += ldw;
                    if (scale) {
                        scale += nb;
                        if (row < w.rows) inv = inverse_pow2(__ldg(row_pow2 + row));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i >= n) break;
            uint32_t v[4];
#pragma unroll
            for (int h = 0; h < H; ++h)
                decode_weights<K, N, CODE>(hi[i][h], lo[i][h], down[i][h], mask, sm, sc[i][h], v + N / 2 * h);
            // ldw is cols rounded up to 8: a lane's eight columns are all stored (those
            // behind the last are padding that nothing reads) or none is
            if (to[i] && TCQ_IN_BOUNDS(to[i] - out + 7, w.rows * ldw))
                *reinterpret_cast<uint4*>(to[i]) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        left -= n;
    }
}

template <int K, int CODE, int N, bool T32>
cudaError_t launch(const CodedMatrix& w, void* out, long long ldw, const float* row_pow2, int num_sms,
                   cudaStream_t stream)
{
    const size_t smem = table_bytes(CODE, w.L);
    cudaError_t e = cudaFuncSetAttribute(decode16_kernel<K, CODE, N, T32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const long long units = (w.cols + kUnit - 1) / kUnit * w.rows;
    const long long need = (units + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = (int)(need < num_sms ? need : num_sms);
    return launch_pdl(decode16_kernel<K, CODE, N, T32>, dim3(grid), dim3(kThreads), smem, stream, w.scale != nullptr, w,
                      static_cast<uint16_t*>(out), ldw, row_pow2);
}

template <int CODE>
cudaError_t launch_k(const CodedMatrix& w, void* out, long long ldw, const float* row_pow2, int num_sms,
                     cudaStream_t stream)
{
#define TCQ_DECODE16(KK)                                                                     \
    case KK:                                                                                 \
        return w.T % 32 == 0  ? launch<KK, CODE, 8, true>(w, out, ldw, row_pow2, num_sms, stream)  \
               : w.T % 8 == 0 ? launch<KK, CODE, 8, false>(w, out, ldw, row_pow2, num_sms, stream) \
                              : launch<KK, CODE, 4, false>(w, out, ldw, row_pow2, num_sms, stream);
    switch (w.K) {
        TCQ_DECODE16(1)
        TCQ_DECODE16(2)
        TCQ_DECODE16(3)
        TCQ_DECODE16(4)
    default: return cudaErrorInvalidValue;
    }
#undef TCQ_DECODE16
}

}  // namespace

cudaError_t launch_row_pow2(const CodedMatrix& w, float* row_pow2, cudaStream_t stream)
{
    row_pow2_kernel<<<(unsigned)((w.rows + 7) / 8), 256, 0, stream>>>(w.scale, w.rows, w.cols / w.T, row_pow2);
    return cudaGetLastError();
}

cudaError_t launch_decode16(const CodedMatrix& w, void* out, long long ldw, float* row_pow2, int num_sms,
                            cudaStream_t stream)
{
    if (w.scale) {
        const cudaError_t e = launch_row_pow2(w, row_pow2, stream);
        if (e != cudaSuccess) return e;
    }
    switch (w.cb_f16) {
    case kMadCodebook: return launch_k<kCode16Mad>(w, out, ldw, row_pow2, num_sms, stream);
    case 1: return launch_k<kCode16F16>(w, out, ldw, row_pow2, num_sms, stream);
    default: return launch_k<kCode16F32>(w, out, ldw, row_pow2, num_sms, stream);
    }
}

}  // namespace tcq
