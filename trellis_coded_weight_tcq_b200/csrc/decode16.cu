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
// two stream words, one 16-byte store per lane.  Table lookups at random
// shared-memory addresses bound it (as in the decoder), then the 2 bytes per weight
// written.
#include "codes.cuh"
#include "decode16.cuh"
#include "gemm.cuh"

namespace tcq {

namespace {

constexpr int kThreads = 1024;
constexpr int kUnit = 256;  // columns per warp step
constexpr int kAhead = 4;   // steps whose words are loaded together

template <int K, int CODE>
__global__ void __launch_bounds__(kThreads, 1) decode16_kernel(CodedMatrix w, uint16_t* out, long long ldw,
                                                               float* row_pow2)
{
    extern __shared__ __align__(16) unsigned char sm[];
    stage_table<CODE>(sm, w.cb, w.cb_f16, w.L);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const long long nb = w.cols / w.T;
    const long long upr = (w.cols + kUnit - 1) / kUnit;
    const long long units = upr * w.rows;
    const long long nwarps = ((long long)gridDim.x * blockDim.x) >> 5;
    const long long me = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const uint32_t mask = (1u << w.L) - 1u;
    // contiguous runs of units, so that a row's scale power is found once per run
    const long long u0 = units * me / nwarps, u1 = units * (me + 1) / nwarps;
    long long row = -1;
    float inv = 1.f;
    const bool eights = w.T % 8 == 0;
    const int tshift = (w.T & (w.T - 1)) == 0 ? __ffs(w.T) - 1 : -1;
    for (long long u = u0; u < u1; u += kAhead) {
        uint32_t hi[kAhead][2], lo[kAhead][2];
        float sc[kAhead][2];
        int q[kAhead][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (u + i >= u1) break;
            const long long r = (u + i) / upr;
            const long long c = (u + i - r * upr) * kUnit + 8 * lane;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && eights) break;
                const long long ch = c + 4 * h;
                hi[i][h] = lo[i][h] = 0u;
                sc[i][h] = 0.f;
                q[i][h] = 0;
                if (ch < w.cols) {
                    const long long j = tshift >= 0 ? ch >> tshift : ch / w.T;
                    const long long b = r * nb + j;
                    const int t0 = (int)(ch - j * w.T);
                    q[i][h] = t0;
                    const int e = (K * (t0 + (eights ? 8 : 4)) - 1) >> 5;  // word the last window ends in
                    if (TCQ_IN_BOUNDS(b, w.rows * nb)) {
                        const uint32_t* wb = w.bits + b * w.W;
                        hi[i][h] = e > 0 ? __ldg(wb + e - 1) : __ldg(w.start_state + b);
                        lo[i][h] = __ldg(wb + e);
                        sc[i][h] = w.scale ? __ldg(w.scale + b) : 1.f;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (u + i >= u1) break;
            const long long r = (u + i) / upr;
            const long long c = (u + i - r * upr) * kUnit + 8 * lane;
            if (w.scale && r != row) {  // the same in every lane
                row = r;
                uint32_t top = 0u;
                for (long long j = lane; j < nb; j += 32) top = max(top, finite_magnitude(__ldg(w.scale + r * nb + j)));
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int p = power_above(top);
                inv = pow2_clamped(-p);
                if (lane == 0) row_pow2[r] = pow2_clamped(p);
            }
            uint32_t v[4];
            if (eights) {
                uint32_t s[8];
                windows<K, 8>(hi[i][0], lo[i][0], q[i][0], mask, s);
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    v[e / 2] = weight_pair<CODE>(s[e], s[e + 1], sm, sc[i][0] * inv);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t s[4];
                    windows<K, 4>(hi[i][h], lo[i][h], q[i][h], mask, s);
                    v[2 * h] = weight_pair<CODE>(s[0], s[1], sm, sc[i][h] * inv);
                    v[2 * h + 1] = weight_pair<CODE>(s[2], s[3], sm, sc[i][h] * inv);
                }
            }
            // ldw is cols rounded up to 8: a lane's eight columns are all stored (those
            // behind the last are padding that nothing reads) or none is
            if (c < w.cols && TCQ_IN_BOUNDS(r * ldw + c + 7, w.rows * ldw))
                *reinterpret_cast<uint4*>(out + r * ldw + c) = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

template <int K, int CODE>
cudaError_t launch(const CodedMatrix& w, void* out, long long ldw, float* row_pow2, int num_sms, cudaStream_t stream)
{
    const size_t smem = table_bytes(CODE, w.L);
    cudaError_t e = cudaFuncSetAttribute(decode16_kernel<K, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const long long units = (w.cols + kUnit - 1) / kUnit * w.rows;
    const long long need = (units + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = (int)(need < num_sms ? need : num_sms);
    decode16_kernel<K, CODE><<<grid, kThreads, smem, stream>>>(w, static_cast<uint16_t*>(out), ldw, row_pow2);
    return cudaGetLastError();
}

template <int CODE>
cudaError_t launch_k(const CodedMatrix& w, void* out, long long ldw, float* row_pow2, int num_sms, cudaStream_t stream)
{
    switch (w.K) {
    case 1: return launch<1, CODE>(w, out, ldw, row_pow2, num_sms, stream);
    case 2: return launch<2, CODE>(w, out, ldw, row_pow2, num_sms, stream);
    case 3: return launch<3, CODE>(w, out, ldw, row_pow2, num_sms, stream);
    default: return launch<4, CODE>(w, out, ldw, row_pow2, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_decode16(const CodedMatrix& w, void* out, long long ldw, float* row_pow2, int num_sms,
                            cudaStream_t stream)
{
    switch (w.cb_f16) {
    case kMadCodebook: return launch_k<kCode16Mad>(w, out, ldw, row_pow2, num_sms, stream);
    case 1: return launch_k<kCode16F16>(w, out, ldw, row_pow2, num_sms, stream);
    default: return launch_k<kCode16F32>(w, out, ldw, row_pow2, num_sms, stream);
    }
}

}  // namespace tcq
